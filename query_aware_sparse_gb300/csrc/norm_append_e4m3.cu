#include "norm_append.cuh"

namespace quest {

cudaError_t launch_norm_append_e4m3(const NormAppendArgs& p, dim3 grid, int sms, cudaStream_t s) {
  if (p.a.summary_fp8)
    return p.a.head_dim == 128 ? launch_norm_append_t<__half, 128, true, true>(p, grid, sms, s)
                               : launch_norm_append_t<__half, 64, true, true>(p, grid, sms, s);
  return p.a.head_dim == 128 ? launch_norm_append_t<__half, 128, true, false>(p, grid, sms, s)
                             : launch_norm_append_t<__half, 64, true, false>(p, grid, sms, s);
}

}  // namespace quest
