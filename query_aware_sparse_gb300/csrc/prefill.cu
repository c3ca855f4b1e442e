// Prompt attention: the new tokens of each request over its paged cache. Plan,
// tensor maps and dispatch; fp16 on the tensor cores (prefill_mma.cuh), fp32 on
// FMA (prefill_f32.cu).
#include "internal.h"
#include "prefill_mma.cuh"
#include "tmap.h"

namespace quest {

#define QUEST_PREFILL_VARIANT(d, t) \
  cudaError_t launch_prefill_f16_d##d##_t##t(const PrefillMaps& maps, const PrefillArgs& p, cudaStream_t s);
QUEST_PREFILL_VARIANT(64, 1)
QUEST_PREFILL_VARIANT(64, 2)
QUEST_PREFILL_VARIANT(128, 1)
QUEST_PREFILL_VARIANT(128, 2)
#undef QUEST_PREFILL_VARIANT
cudaError_t launch_prefill_f32(const PrefillArgs& p, cudaStream_t s);

namespace {

struct Plan {
  int tiles, blocks, splits, near_heads;
  size_t lse_at, bytes;               // of the partial results in the workspace
};

Plan plan_prefill(int32_t batch, int32_t n_q, int32_t nnz, int32_t h_kv, int32_t group,
                  int32_t head_dim, int32_t page_size, int32_t dtype) {
  Plan p{1, 0, 1, h_kv, 0, 16};
  if (n_q == 0 || batch == 0) return p;
  // fp16: two tiles where the requests' rows fill more than one on average
  const bool f16 = dtype == QUEST_F16;
  if (f16 && (long long)n_q * group > 128LL * batch) p.tiles = 2;
  const int rows = f16 ? p.tiles * 128 : 64, keys = p.tiles == 2 ? 128 : 64;
  const int per_sm = p.tiles == 2 ? 1 : 2;             // CTAs an SM holds
  const int tokens = rows / group;
  const long long blocks = (long long)n_q / tokens + batch;
  p.blocks = (int)(blocks < n_q ? blocks : n_q);
  // Many row blocks read the same keys: as many KV heads at a time as fit half
  // of the L2 (16384 tokens of 32 heads: 1.52 ms with all of them, 1.43 with
  // one by one). Otherwise all heads side by side, longest rows first.
  const long long head_bytes = (long long)nnz * page_size * head_dim * (f16 ? 4 : 8);
  if (p.blocks >= 4LL * batch && head_bytes * h_kv > 64ll << 20)
    p.near_heads = head_bytes > 64ll << 20 ? 1 : (int)((64ll << 20) / head_bytes);
  // Too few CTAs for the device: cut each one's keys. Ragged requests get
  // twice the CTAs that run at once, so that the long ones even out.
  const long long units = (long long)p.blocks * h_kv;
  const long long want = (long long)sm_count() * per_sm * (batch > 1 ? 2 : 1);
  const long long key_blocks = ((long long)nnz * page_size / batch + keys - 1) / keys;
  if (units < want) {
    long long s = (want + units - 1) / units;
    if (s > (key_blocks + 1) / 2) s = (key_blocks + 1) / 2;
    if (s > 1) p.splits = (int)s;
  }
  if (p.splits > 1) {
    const size_t all = (size_t)p.splits * n_q * h_kv * group;
    p.lse_at = all * head_dim * sizeof(float);
    p.bytes = p.lse_at + all * sizeof(float);
  }
  return p;
}

PrefillArgs prefill_args(const DenseArgs& a, const Plan& plan) {
  PrefillArgs p{};
  p.a = a;
  p.blocks = plan.blocks;
  p.splits = plan.splits;
  p.near_heads = plan.near_heads;
  p.part_o = static_cast<float*>(a.workspace);
  p.part_lse = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + plan.lse_at);
  p.wait_limit = wait_limit();
  return p;
}

cudaError_t launch_f16(const PrefillArgs& p, int tiles, cudaStream_t s) {
  const DenseArgs& a = p.a;
  PrefillMaps maps;
  const cuuint64_t d = a.head_dim, hq = (cuuint64_t)a.h_kv * a.group;
  // queries: a box is one tile's tokens with their group's heads, 64 dims
  const cuuint64_t q_dims[3] = {d, hq, (cuuint64_t)a.n_q}, q_strides[2] = {d * 2, hq * d * 2};
  const cuuint32_t q_box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)(128 / a.group)};
  // pools: a box is one page of one KV head, 64 dims
  if (!encode_map(&maps.q, a.dtype, a.q, 3, q_dims, q_strides, q_box) ||
      !encode_map(&maps.out, a.dtype, a.out, 3, q_dims, q_strides, q_box) ||
      !encode_pool(&maps.k, a, a.k_pool, a.page_size) || !encode_pool(&maps.v, a, a.v_pool, a.page_size))
    return cudaErrorInvalidValue;
  if (a.head_dim == 128)
    return tiles == 2 ? launch_prefill_f16_d128_t2(maps, p, s) : launch_prefill_f16_d128_t1(maps, p, s);
  return tiles == 2 ? launch_prefill_f16_d64_t2(maps, p, s) : launch_prefill_f16_d64_t1(maps, p, s);
}

}  // namespace

size_t prefill_workspace(int32_t batch, int32_t n_q, int32_t nnz, int32_t h_kv, int32_t group,
                         int32_t head_dim, int32_t page_size, int32_t dtype) {
  return plan_prefill(batch, n_q, nnz, h_kv, group, head_dim, page_size, dtype).bytes;
}

cudaError_t launch_prefill(const DenseArgs& a, cudaStream_t s) {
  const Plan plan = plan_prefill(a.batch, a.n_q, a.nnz, a.h_kv, a.group, a.head_dim, a.page_size, a.dtype);
  const PrefillArgs p = prefill_args(a, plan);
  return a.dtype == QUEST_F16 ? launch_f16(p, plan.tiles, s) : launch_prefill_f32(p, s);
}

}  // namespace quest
