// C ABI of the dense-layer operators: host-side validation and dispatch.
#include <math.h>

#include "dense.h"
#include "internal.h"

namespace {

using quest::aligned16;
using quest::check_cache;
using quest::check_mods;
using quest::check_pages;
using quest::launched;
using quest::valid_group;
using quest::valid_stride;

bool valid_shape(int32_t h_kv, int32_t group, int32_t head_dim, int32_t page_size, int32_t dtype) {
  return h_kv > 0 && valid_group(group) && (head_dim == 64 || head_dim == 128) &&
         (page_size == 16 || page_size == 32) && (dtype == QUEST_F16 || dtype == QUEST_F32);
}

// The attention kernels name a pool's rows (one token of one KV head) by the
// signed 32-bit coordinate of a tensor map.
bool addressable(const quest_cache* c) {
  return (int64_t)c->n_phys * c->h_kv <= INT32_MAX / c->page_size;
}

quest::DenseArgs dense_args(const quest_cache* cache, const quest_pages* pages, const void* q,
                            int32_t group, const quest_score_mods* mods, void* out, float* lse,
                            float sm_scale, void* workspace) {
  quest::DenseArgs a{};
  a.k_pool = cache->k_pool; a.v_pool = cache->v_pool; a.q = q;
  a.page_indptr = pages->page_indptr; a.page_indices = pages->page_indices;
  a.seq_lens = pages->seq_lens;
  if (mods) {
    a.slopes = mods->alibi_slopes; a.doc_starts = mods->doc_starts;
    a.prefix_lens = mods->prefix_lens; a.softcap = mods->softcap; a.window = mods->window;
  }
  a.out = out; a.lse = lse; a.workspace = workspace;
  a.batch = pages->batch; a.nnz = pages->nnz; a.n_phys = cache->n_phys; a.h_kv = cache->h_kv;
  a.group = group; a.page_size = cache->page_size; a.head_dim = cache->head_dim;
  a.dtype = cache->dtype;
  a.scale = sm_scale > 0.f ? sm_scale : 1.0f / sqrtf((float)cache->head_dim);
  a.test_fault = quest::test_fault_mode();
  a.err = quest::error_word_ptr();
  return a;
}

}  // namespace

extern "C" {

quest_status quest_rope_append_kv(const quest_cache* cache, const quest_pages* pages,
                                  const quest_rope* rope, const void* q, const void* k_new,
                                  const void* v_new, int64_t q_stride, int64_t k_stride,
                                  int64_t v_stride, int32_t n_new, int32_t group,
                                  const int32_t* append_indptr, const int32_t* seq_lens_before,
                                  void* q_out, void* stream) {
  quest_status st = check_cache(cache);
  if (st != QUEST_OK) return st;
  if ((st = check_pages(pages, false)) != QUEST_OK) return st;
  if (!valid_group(group)) return QUEST_ERR_UNSUPPORTED;
  if (!rope || n_new < 0) return QUEST_ERR_INVALID_ARG;
  if (rope->rotary_dim < 16 || rope->rotary_dim > cache->head_dim || rope->rotary_dim % 16 != 0)
    return QUEST_ERR_UNSUPPORTED;
  if (rope->interleaved != 0 && rope->interleaved != 1) return QUEST_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return QUEST_ERR_INVALID_ARG;
  const int64_t kv_row = (int64_t)cache->h_kv * cache->head_dim, q_row = kv_row * group;
  if (!valid_stride(k_stride, kv_row, cache->dtype) || !valid_stride(v_stride, kv_row, cache->dtype) ||
      (q && !valid_stride(q_stride, q_row, cache->dtype)))
    return QUEST_ERR_INVALID_ARG;
  if (q == q_out && q && q_stride != q_row) return QUEST_ERR_INVALID_ARG;
  if (pages->batch == 0 || n_new == 0) return QUEST_OK;
  if (!k_new || !v_new || !append_indptr || !seq_lens_before || !rope->inv_freq)
    return QUEST_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(q) || !aligned16(q_out) ||
      (reinterpret_cast<uintptr_t>(rope->inv_freq) & 7u) != 0)
    return QUEST_ERR_INVALID_ARG;
  quest::RopeAppendArgs a{};
  a.k_pool = cache->k_pool; a.v_pool = cache->v_pool; a.summary = cache->summary;
  a.q = q; a.k_new = k_new; a.v_new = v_new; a.q_out = q_out;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.inv_freq = rope->inv_freq; a.positions = rope->positions;
  a.page_indptr = pages->page_indptr; a.page_indices = pages->page_indices;
  a.append_indptr = append_indptr; a.seq_lens_before = seq_lens_before;
  a.batch = pages->batch; a.nnz = pages->nnz; a.n_new = n_new; a.n_phys = cache->n_phys;
  a.h_kv = cache->h_kv; a.group = group; a.page_size = cache->page_size;
  a.head_dim = cache->head_dim; a.dtype = cache->dtype; a.summary_fp8 = cache->summary_fp8;
  a.rotary_dim = rope->rotary_dim; a.interleaved = rope->interleaved;
  a.err = quest::error_word_ptr();
  if (!a.err) return QUEST_ERR_CUDA;
  return launched(quest::launch_rope_append(a, static_cast<cudaStream_t>(stream)));
}

size_t quest_dense_decode_workspace_size(int32_t batch, int32_t nnz, int32_t h_kv, int32_t group,
                                         int32_t head_dim, int32_t page_size, int32_t dtype) {
  if (batch <= 0 || batch > quest::kDecodeMaxBatch || nnz < 0 ||
      !valid_shape(h_kv, group, head_dim, page_size, dtype))
    return 0;
  return quest::dense_decode_workspace(batch, nnz, h_kv, group, head_dim, page_size, dtype);
}

quest_status quest_dense_decode_attn(const quest_cache* cache, const quest_pages* pages,
                                     const void* q, int32_t group, const quest_score_mods* mods,
                                     float* out, float* lse, float sm_scale, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  quest_status st = check_cache(cache);
  if (st != QUEST_OK) return st;
  if ((st = check_pages(pages, true)) != QUEST_OK) return st;
  if (!valid_group(group)) return QUEST_ERR_UNSUPPORTED;
  if ((st = check_mods(mods)) != QUEST_OK) return st;
  if (!addressable(cache)) return QUEST_ERR_UNSUPPORTED;
  if (pages->batch == 0) return QUEST_OK;
  if (pages->batch > quest::kDecodeMaxBatch) return QUEST_ERR_UNSUPPORTED;
  if (!q || !out || !aligned16(q) || !aligned16(out)) return QUEST_ERR_INVALID_ARG;
  const size_t need = quest::dense_decode_workspace(pages->batch, pages->nnz, cache->h_kv, group,
                                                    cache->head_dim, cache->page_size, cache->dtype);
  if (!workspace || workspace_bytes < need || !aligned16(workspace)) return QUEST_ERR_WORKSPACE;
  quest::DenseArgs a = dense_args(cache, pages, q, group, mods, out, lse, sm_scale, workspace);
  a.n_q = pages->batch;
  if (!a.err) return QUEST_ERR_CUDA;
  return launched(quest::launch_dense_decode(a, static_cast<cudaStream_t>(stream)));
}

size_t quest_prefill_workspace_size(int32_t batch, int32_t n_q, int32_t nnz, int32_t h_kv,
                                    int32_t group, int32_t head_dim, int32_t page_size,
                                    int32_t dtype) {
  if (batch <= 0 || n_q < 0 || nnz < 0 || !valid_shape(h_kv, group, head_dim, page_size, dtype))
    return 0;
  return quest::prefill_workspace(batch, n_q, nnz, h_kv, group, head_dim, page_size, dtype);
}

quest_status quest_prefill_attn(const quest_cache* cache, const quest_pages* pages, const void* q,
                                int32_t group, const int32_t* q_indptr, int32_t n_q,
                                const quest_score_mods* mods, void* out, float* lse,
                                float sm_scale, void* workspace, size_t workspace_bytes,
                                void* stream) {
  quest_status st = check_cache(cache);
  if (st != QUEST_OK) return st;
  if ((st = check_pages(pages, true)) != QUEST_OK) return st;
  if (!valid_group(group)) return QUEST_ERR_UNSUPPORTED;
  if ((st = check_mods(mods)) != QUEST_OK) return st;
  if (!addressable(cache)) return QUEST_ERR_UNSUPPORTED;
  if (n_q < 0) return QUEST_ERR_INVALID_ARG;
  if (pages->batch == 0 || n_q == 0) return QUEST_OK;
  if (!q || !q_indptr || !out || !aligned16(q) || !aligned16(out)) return QUEST_ERR_INVALID_ARG;
  const size_t need = quest::prefill_workspace(pages->batch, n_q, pages->nnz, cache->h_kv, group,
                                               cache->head_dim, cache->page_size, cache->dtype);
  if (!workspace || workspace_bytes < need || !aligned16(workspace)) return QUEST_ERR_WORKSPACE;
  quest::DenseArgs a = dense_args(cache, pages, q, group, mods, out, lse, sm_scale, workspace);
  a.q_indptr = q_indptr; a.n_q = n_q;
  if (!a.err) return QUEST_ERR_CUDA;
  return launched(quest::launch_prefill(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
