// Host-side interfaces of the dense-layer operators: the rotating append
// (rope_append.cu), dense decode attention (dense_decode.cu) and prompt
// attention (prefill.cu), behind dense_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/quest.h"

namespace quest {

struct RopeAppendArgs {
  void* k_pool; void* v_pool; void* summary;
  const void* q; const void* k_new; const void* v_new; void* q_out;
  int64_t q_stride, k_stride, v_stride;       // elements between tokens
  const double* inv_freq; const int32_t* positions;
  const int32_t* page_indptr; const int32_t* page_indices;
  const int32_t* append_indptr; const int32_t* seq_lens_before;
  int32_t batch, nnz, n_new, n_phys, h_kv, group, page_size, head_dim, dtype;
  int32_t summary_fp8, rotary_dim, interleaved;
  int32_t heads_per_cta;                      // KV heads one CTA takes (set by the launch)
  unsigned* err;
};
cudaError_t launch_rope_append(const RopeAppendArgs& a, cudaStream_t s);

// Attention over the page table itself: n_q query rows, q_indptr null for one
// row per request.
struct DenseArgs {
  const void* k_pool; const void* v_pool; const void* q;
  const int32_t* page_indptr; const int32_t* page_indices; const int32_t* seq_lens;
  const int32_t* q_indptr;
  const float* slopes; const int32_t* doc_starts; const int32_t* prefix_lens;
  float softcap; int32_t window;              // 0 = none
  void* out; float* lse;
  void* workspace;
  int32_t batch, nnz, n_q, n_phys, h_kv, group, page_size, head_dim, dtype;
  float scale;
  int32_t test_fault;                         // 2: a copy of the first CTA never completes (tests)
  unsigned* err;
};
constexpr int32_t kDecodeMaxBatch = 1 << 19;  // its running sums stay in shared memory
size_t dense_decode_workspace(int32_t batch, int32_t nnz, int32_t h_kv, int32_t group,
                              int32_t head_dim, int32_t page_size, int32_t dtype);
cudaError_t launch_dense_decode(const DenseArgs& a, cudaStream_t s);
size_t prefill_workspace(int32_t batch, int32_t n_q, int32_t nnz, int32_t h_kv, int32_t group,
                         int32_t head_dim, int32_t page_size, int32_t dtype);
cudaError_t launch_prefill(const DenseArgs& a, cudaStream_t s);

}  // namespace quest
