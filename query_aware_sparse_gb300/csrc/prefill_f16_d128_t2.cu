// Prompt attention, fp16, head dim 128, 2 row tiles per CTA.
#include "prefill_mma.cuh"

namespace quest {

cudaError_t launch_prefill_f16_d128_t2(const PrefillMaps& maps, const PrefillArgs& p, cudaStream_t s) {
  return launch_prefill_mma_t<128, 2>(maps, p, s);
}

}  // namespace quest
