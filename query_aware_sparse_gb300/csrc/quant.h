// Host-side interfaces of the normed append and of the E4M3 cache: append
// (norm_append*.cu), read-back (quant_read.cu) and decode attention
// (quant_decode.cu), behind quant_api.cu.
#pragma once

#include "dense.h"

namespace quest {

// a: as for the rotating append, with rotary_dim 0 for keys that are not
// rotated here. e4m3: a.k_pool holds records, a.v_pool is not used.
struct NormAppendArgs {
  RopeAppendArgs a;
  const float* q_weight; const float* k_weight;   // null: not normed
  int32_t q_per_head, k_per_head;                 // a weight row per head
  float eps;
};
cudaError_t launch_norm_append(const NormAppendArgs& p, bool e4m3, cudaStream_t s);
// Per store, element type and head dim (norm_append_<name>.cu).
#define QUEST_NORM_APPEND(name) \
  cudaError_t launch_norm_append_##name(const NormAppendArgs& p, dim3 grid, int sms, cudaStream_t s);
QUEST_NORM_APPEND(e4m3_d64)
QUEST_NORM_APPEND(e4m3_d128)
QUEST_NORM_APPEND(f16_d64)
QUEST_NORM_APPEND(f16_d128)
QUEST_NORM_APPEND(f32)
#undef QUEST_NORM_APPEND

struct QuantReadArgs {
  const uint8_t* pool; void* k_out; void* v_out;
  const int32_t* page_indptr; const int32_t* page_indices; const int32_t* seq_lens;
  const int32_t* dst_indices;                     // null: entry e goes to page e
  int32_t batch, nnz, n_phys, n_dst, h_kv, page_size, head_dim;
  unsigned* err;
};
cudaError_t launch_quant_read(const QuantReadArgs& a, cudaStream_t s);

// a.k_pool holds records; sel_logical null: the page table's pages.
size_t quant_decode_workspace(int32_t batch, int32_t h_kv, int32_t group, int32_t head_dim);
cudaError_t launch_quant_decode(const DenseArgs& a, const int32_t* sel_logical, const int32_t* sel_phys,
                                int32_t k, cudaStream_t s);

}  // namespace quest
