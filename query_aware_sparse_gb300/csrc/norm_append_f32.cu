#include "norm_append.cuh"

namespace quest {

cudaError_t launch_norm_append_f32(const NormAppendArgs& p, dim3 grid, int sms, cudaStream_t s) {
  return p.a.head_dim == 128 ? launch_norm_append_t<float, 128, false, false>(p, grid, sms, s)
                             : launch_norm_append_t<float, 64, false, false>(p, grid, sms, s);
}

}  // namespace quest
