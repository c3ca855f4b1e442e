#include "norm_append.cuh"

namespace quest {

cudaError_t launch_norm_append_f16_d64(const NormAppendArgs& p, dim3 grid, int sms, cudaStream_t s) {
  return p.a.summary_fp8 ? launch_norm_append_t<__half, 64, false, true>(p, grid, sms, s)
                         : launch_norm_append_t<__half, 64, false, false>(p, grid, sms, s);
}

}  // namespace quest
