// Prompt attention, fp16, head dim 64, 2 row tiles per CTA.
#include "prefill_mma.cuh"

namespace quest {

cudaError_t launch_prefill_f16_d64_t2(const PrefillMaps& maps, const PrefillArgs& p, cudaStream_t s) {
  return launch_prefill_mma_t<64, 2>(maps, p, s);
}

}  // namespace quest
