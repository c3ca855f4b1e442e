// Prompt attention, fp16, head dim 128, 1 row tile per CTA.
#include "prefill_mma.cuh"

namespace quest {

cudaError_t launch_prefill_f16_d128_t1(const PrefillMaps& maps, const PrefillArgs& p, cudaStream_t s) {
  return launch_prefill_mma_t<128, 1>(maps, p, s);
}

}  // namespace quest
