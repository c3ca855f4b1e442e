// Prompt attention: the new tokens of each request over its paged cache.
#include "dense_rows.cuh"

namespace quest {

size_t prefill_workspace(int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t) {
  return 16;
}

cudaError_t launch_prefill(const DenseArgs& a, cudaStream_t s) {
  const dim3 grid(a.n_q, a.h_kv * a.group);
  if (a.dtype == QUEST_F16) {
    if (a.head_dim == 128) dense_rows_kernel<__half, __half, 128><<<grid, kRowThreads, 0, s>>>(a);
    else dense_rows_kernel<__half, __half, 64><<<grid, kRowThreads, 0, s>>>(a);
  } else {
    if (a.head_dim == 128) dense_rows_kernel<float, float, 128><<<grid, kRowThreads, 0, s>>>(a);
    else dense_rows_kernel<float, float, 64><<<grid, kRowThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace quest
