// C ABI of the normed append and of the E4M3 cache: host-side validation and
// dispatch.
#include <float.h>

#include "internal.h"
#include "quant.h"

namespace {

using quest::aligned16;
using quest::check_cache;
using quest::check_mods;
using quest::check_pages;
using quest::launched;
using quest::valid_group;
using quest::valid_stride;

quest_status check_quant(const quest_quant_cache* c) {
  if (!c || !c->pool || !c->summary || c->n_phys <= 0 || c->h_kv <= 0) return QUEST_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return QUEST_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32) return QUEST_ERR_UNSUPPORTED;
  if (c->summary_fp8 != 0 && c->summary_fp8 != 1) return QUEST_ERR_INVALID_ARG;
  if (!aligned16(c->pool) || !aligned16(c->summary)) return QUEST_ERR_INVALID_ARG;
  return QUEST_OK;
}

// The queries, keys and values of an append and what is done to them; `a` has
// the cache's sizes. QUEST_OK with a.n_new 0: nothing to do.
quest_status take_append(quest::NormAppendArgs& p, const quest_pages* pages, const quest_rope* rope,
                         const quest_qk_norm* norm, const void* q, const void* k_new, const void* v_new,
                         int64_t q_stride, int64_t k_stride, int64_t v_stride, int32_t n_new, int32_t group,
                         const int32_t* append_indptr, const int32_t* seq_lens_before, void* q_out) {
  quest::RopeAppendArgs& a = p.a;
  quest_status st = check_pages(pages, false);
  if (st != QUEST_OK) return st;
  if (!valid_group(group)) return QUEST_ERR_UNSUPPORTED;
  if (n_new < 0) return QUEST_ERR_INVALID_ARG;
  if (rope) {
    if (rope->rotary_dim < 16 || rope->rotary_dim > a.head_dim || rope->rotary_dim % 16 != 0)
      return QUEST_ERR_UNSUPPORTED;
    if (rope->interleaved != 0 && rope->interleaved != 1) return QUEST_ERR_INVALID_ARG;
  }
  if (norm) {
    if (!(norm->eps >= FLT_MIN && norm->eps <= FLT_MAX)) return QUEST_ERR_INVALID_ARG;
    if ((norm->q_per_head & ~1) || (norm->k_per_head & ~1)) return QUEST_ERR_INVALID_ARG;
    if (!aligned16(norm->q_weight) || !aligned16(norm->k_weight)) return QUEST_ERR_INVALID_ARG;
  }
  if ((q == nullptr) != (q_out == nullptr)) return QUEST_ERR_INVALID_ARG;
  if (q && !rope && !(norm && norm->q_weight)) return QUEST_ERR_INVALID_ARG;
  const int64_t kv_row = (int64_t)a.h_kv * a.head_dim, q_row = kv_row * group;
  if (!valid_stride(k_stride, kv_row, a.dtype) || !valid_stride(v_stride, kv_row, a.dtype) ||
      (q && !valid_stride(q_stride, q_row, a.dtype)))
    return QUEST_ERR_INVALID_ARG;
  if (q == q_out && q && q_stride != q_row) return QUEST_ERR_INVALID_ARG;
  if (pages->batch == 0 || n_new == 0) return QUEST_OK;
  if (!k_new || !v_new || !append_indptr || !seq_lens_before || (rope && !rope->inv_freq))
    return QUEST_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(q) || !aligned16(q_out) ||
      (rope && (reinterpret_cast<uintptr_t>(rope->inv_freq) & 7u) != 0))
    return QUEST_ERR_INVALID_ARG;
  a.q = q; a.k_new = k_new; a.v_new = v_new; a.q_out = q_out;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  if (rope) {
    a.inv_freq = rope->inv_freq; a.positions = rope->positions;
    a.rotary_dim = rope->rotary_dim; a.interleaved = rope->interleaved;
  }
  if (norm) {
    p.q_weight = norm->q_weight; p.k_weight = norm->k_weight;
    p.q_per_head = norm->q_per_head; p.k_per_head = norm->k_per_head; p.eps = norm->eps;
  }
  a.page_indptr = pages->page_indptr; a.page_indices = pages->page_indices;
  a.append_indptr = append_indptr; a.seq_lens_before = seq_lens_before;
  a.batch = pages->batch; a.nnz = pages->nnz; a.group = group; a.n_new = n_new;
  a.err = quest::error_word_ptr();
  return a.err ? QUEST_OK : QUEST_ERR_CUDA;
}

// Sizes that the decode kernels' grids and running sums take.
bool decodable(int32_t batch, int32_t h_kv, int32_t group) {
  return batch <= quest::kDecodeMaxBatch && (int64_t)batch * h_kv * group <= INT32_MAX;
}

quest_status quant_attn(const quest_quant_cache* cache, const quest_pages* pages, const void* q, int32_t group,
                        const int32_t* sel_logical, const int32_t* sel_phys, int32_t k,
                        const quest_score_mods* mods, float* out, float* lse, float sm_scale, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!q || !out || !aligned16(q) || !aligned16(out)) return QUEST_ERR_INVALID_ARG;
  const size_t need = quest::quant_decode_workspace(pages->batch, cache->h_kv, group, cache->head_dim);
  if (!workspace || workspace_bytes < need || !aligned16(workspace)) return QUEST_ERR_WORKSPACE;
  quest::DenseArgs a{};
  a.k_pool = cache->pool; a.q = q;
  a.page_indptr = pages->page_indptr; a.page_indices = pages->page_indices;
  a.seq_lens = pages->seq_lens;
  if (mods) {
    a.slopes = mods->alibi_slopes; a.doc_starts = mods->doc_starts;
    a.prefix_lens = mods->prefix_lens; a.softcap = mods->softcap; a.window = mods->window;
  }
  a.out = out; a.lse = lse; a.workspace = workspace;
  a.batch = pages->batch; a.nnz = pages->nnz; a.n_q = pages->batch; a.n_phys = cache->n_phys;
  a.h_kv = cache->h_kv; a.group = group; a.page_size = cache->page_size;
  a.head_dim = cache->head_dim; a.dtype = QUEST_F16;
  a.scale = sm_scale > 0.f ? sm_scale : 1.0f / sqrtf((float)cache->head_dim);
  a.test_fault = quest::test_fault_mode();
  a.err = quest::error_word_ptr();
  if (!a.err) return QUEST_ERR_CUDA;
  return launched(quest::launch_quant_decode(a, sel_logical, sel_phys, k, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

quest_status quest_norm_rope_append_kv(const quest_cache* cache, const quest_pages* pages,
                                       const quest_rope* rope, const quest_qk_norm* norm, const void* q,
                                       const void* k_new, const void* v_new, int64_t q_stride,
                                       int64_t k_stride, int64_t v_stride, int32_t n_new, int32_t group,
                                       const int32_t* append_indptr, const int32_t* seq_lens_before,
                                       void* q_out, void* stream) {
  quest_status st = check_cache(cache);
  if (st != QUEST_OK) return st;
  if (!norm) return QUEST_ERR_INVALID_ARG;
  quest::NormAppendArgs p{};
  p.a.k_pool = cache->k_pool; p.a.v_pool = cache->v_pool; p.a.summary = cache->summary;
  p.a.n_phys = cache->n_phys; p.a.h_kv = cache->h_kv; p.a.page_size = cache->page_size;
  p.a.head_dim = cache->head_dim; p.a.dtype = cache->dtype; p.a.summary_fp8 = cache->summary_fp8;
  st = take_append(p, pages, rope, norm, q, k_new, v_new, q_stride, k_stride, v_stride, n_new, group,
                   append_indptr, seq_lens_before, q_out);
  if (st != QUEST_OK || p.a.n_new == 0) return st;
  return launched(quest::launch_norm_append(p, false, static_cast<cudaStream_t>(stream)));
}

size_t quest_quant_page_bytes(int32_t page_size, int32_t head_dim) {
  if ((head_dim != 64 && head_dim != 128) || (page_size != 16 && page_size != 32)) return 0;
  return (size_t)2 * page_size * (head_dim + 1);
}

quest_status quest_quant_append_kv(const quest_quant_cache* cache, const quest_pages* pages,
                                   const quest_rope* rope, const quest_qk_norm* norm, const void* q,
                                   const void* k_new, const void* v_new, int64_t q_stride,
                                   int64_t k_stride, int64_t v_stride, int32_t n_new, int32_t group,
                                   const int32_t* append_indptr, const int32_t* seq_lens_before,
                                   void* q_out, void* stream) {
  quest_status st = check_quant(cache);
  if (st != QUEST_OK) return st;
  quest::NormAppendArgs p{};
  p.a.k_pool = cache->pool; p.a.summary = cache->summary;
  p.a.n_phys = cache->n_phys; p.a.h_kv = cache->h_kv; p.a.page_size = cache->page_size;
  p.a.head_dim = cache->head_dim; p.a.dtype = QUEST_F16; p.a.summary_fp8 = cache->summary_fp8;
  st = take_append(p, pages, rope, norm, q, k_new, v_new, q_stride, k_stride, v_stride, n_new, group,
                   append_indptr, seq_lens_before, q_out);
  if (st != QUEST_OK || p.a.n_new == 0) return st;
  return launched(quest::launch_norm_append(p, true, static_cast<cudaStream_t>(stream)));
}

quest_status quest_quant_read_kv(const quest_quant_cache* cache, const quest_pages* pages, void* k_out,
                                 void* v_out, int32_t n_dst, const int32_t* dst_indices, void* stream) {
  quest_status st = check_quant(cache);
  if (st != QUEST_OK) return st;
  if ((st = check_pages(pages, true)) != QUEST_OK) return st;
  if (n_dst < 0) return QUEST_ERR_INVALID_ARG;
  if (pages->batch == 0) return QUEST_OK;
  if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return QUEST_ERR_INVALID_ARG;
  if ((int64_t)pages->nnz * cache->h_kv > (int64_t)INT32_MAX * 8) return QUEST_ERR_UNSUPPORTED;
  quest::QuantReadArgs a{};
  a.pool = static_cast<const uint8_t*>(cache->pool);
  a.k_out = k_out; a.v_out = v_out;
  a.page_indptr = pages->page_indptr; a.page_indices = pages->page_indices; a.seq_lens = pages->seq_lens;
  a.dst_indices = dst_indices;
  a.batch = pages->batch; a.nnz = pages->nnz; a.n_phys = cache->n_phys; a.n_dst = n_dst;
  a.h_kv = cache->h_kv; a.page_size = cache->page_size; a.head_dim = cache->head_dim;
  a.err = quest::error_word_ptr();
  if (!a.err) return QUEST_ERR_CUDA;
  return launched(quest::launch_quant_read(a, static_cast<cudaStream_t>(stream)));
}

size_t quest_quant_decode_workspace_size(int32_t batch, int32_t h_kv, int32_t group, int32_t head_dim,
                                         int32_t page_size) {
  if (batch <= 0 || h_kv <= 0 || !valid_group(group) || !decodable(batch, h_kv, group) ||
      quest_quant_page_bytes(page_size, head_dim) == 0)
    return 0;
  return quest::quant_decode_workspace(batch, h_kv, group, head_dim);
}

quest_status quest_quant_sparse_decode_attn(const quest_quant_cache* cache, const quest_pages* pages,
                                            const void* q, int32_t group, const int32_t* sel_logical,
                                            const int32_t* sel_phys, int32_t k, float* out, float* lse,
                                            float sm_scale, void* workspace, size_t workspace_bytes,
                                            void* stream) {
  quest_status st = check_quant(cache);
  if (st != QUEST_OK) return st;
  if ((st = check_pages(pages, true)) != QUEST_OK) return st;
  if (!valid_group(group) || k < 1) return QUEST_ERR_INVALID_ARG;
  if (pages->batch == 0) return QUEST_OK;
  if (!decodable(pages->batch, cache->h_kv, group)) return QUEST_ERR_UNSUPPORTED;
  if (!sel_logical || !sel_phys) return QUEST_ERR_INVALID_ARG;
  return quant_attn(cache, pages, q, group, sel_logical, sel_phys, k, nullptr, out, lse, sm_scale, workspace,
                    workspace_bytes, stream);
}

quest_status quest_quant_dense_decode_attn(const quest_quant_cache* cache, const quest_pages* pages,
                                           const void* q, int32_t group, const quest_score_mods* mods,
                                           float* out, float* lse, float sm_scale, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  quest_status st = check_quant(cache);
  if (st != QUEST_OK) return st;
  if ((st = check_pages(pages, true)) != QUEST_OK) return st;
  if (!valid_group(group)) return QUEST_ERR_UNSUPPORTED;
  if ((st = check_mods(mods)) != QUEST_OK) return st;
  if (pages->batch == 0) return QUEST_OK;
  if (!decodable(pages->batch, cache->h_kv, group)) return QUEST_ERR_UNSUPPORTED;
  return quant_attn(cache, pages, q, group, nullptr, nullptr, 0, mods, out, lse, sm_scale, workspace,
                    workspace_bytes, stream);
}

}  // extern "C"
