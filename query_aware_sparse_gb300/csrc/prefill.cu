// Prompt attention: the new tokens of each request over its paged cache. Plan,
// tensor maps and dispatch; fp16 on the tensor cores (prefill_mma.cuh), fp32 on
// FMA (prefill_f32.cu).
#include <math.h>

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
  bool chained;
  size_t lse_at, bytes;               // of the partial results in the workspace
};

// Everything the plan knows: sizes, not the requests' lengths (they are on the
// device), so it goes by their mean. window: 0, or the keys a row sees at most.
Plan plan_prefill(int32_t batch, int32_t n_q, int32_t nnz, int32_t h_kv, int32_t group,
                  int32_t head_dim, int32_t page_size, int32_t dtype, int32_t window) {
  Plan p{1, 0, 1, h_kv, false, 0, 16};
  if (n_q == 0 || batch == 0) return p;
  const bool f16 = dtype == QUEST_F16;
  const long long all_keys = (long long)nnz * page_size;
  const double new_keys = (double)n_q / batch;
  double keys = (double)all_keys / batch;
  double seen = keys > new_keys ? keys - new_keys / 2 : keys / 2;   // by a mean row
  // fp16: two row tiles per CTA where the rows fill them and the loop is long.
  // Its loop is 15% faster (16384-token prompt: 1.34 against 1.44 ms), but one
  // tile per CTA hides its start and end behind a second CTA on the SM (2000
  // tokens, 8 KV heads of 4: 42 against 49 us; packed requests of up to 7000
  // tokens: 130 against 172 us).
  if (f16 && new_keys * group > 128 && seen >= 4096) p.tiles = 2;
  if (window > 0) {                                    // of a row block, then
    const double most = (double)window + p.tiles * 128 / group;
    if (keys > most) keys = most;
    if (seen > most) seen = most;
  }
  const int rows = p.tiles * 128, block = p.tiles == 2 ? 128 : 64;
  const int tokens = rows / group;
  const long long blocks = (long long)n_q / tokens + batch;
  p.blocks = (int)(blocks < n_q ? blocks : n_q);
  // Many row blocks read the same keys: as many KV heads at a time as fit half
  // of the L2 (16384 tokens of 32 heads: 1.52 ms with all of them, 1.43 with
  // one by one). Otherwise all heads side by side, longest rows first.
  const long long head_bytes = all_keys * head_dim * (f16 ? 4 : 8);
  if (p.blocks >= 4LL * batch && head_bytes * h_kv > 64ll << 20)
    p.near_heads = head_bytes > 64ll << 20 ? 1 : (int)((64ll << 20) / head_bytes);
  // Cut each CTA's keys into `splits` parts where that fills the device better
  // than it costs: a part's results are written, read and joined (about 7 TB/s
  // and 4 us), and every wave of CTAs starts and ends (5 us; 2 where two CTAs
  // share an SM). us of a CTA's key block, measured: two tiles 1.24 for 128
  // keys, one 0.71 for 64 (two CTAs per SM), fp32 14 (D = 128). A 512-token
  // chunk of 32768 takes 335 us uncut, 186 in 2, 199 in 4, 223 in 8 parts.
  const double block_us = f16 ? (p.tiles == 2 ? 1.24 : 0.71) : 14.0 * head_dim / 128;
  const double start_us = p.tiles == 2 ? 5 : 2;
  const double slots = (double)sm_count() * (f16 && p.tiles == 1 ? 2 : 1);
  const long long full = ((long long)n_q + tokens - 1) / tokens;
  const double units = (double)(full > batch ? full : batch) * h_kv;
  const double mean_us = seen / block * block_us;
  const bool even = batch == 1 && new_keys * 4 < keys;     // CTAs of about one length
  // the longest: of one request known, of several taken as three times the mean
  const double longest = batch == 1 || even ? 1 : batch < 3 ? batch : 3;
  const double most_us = even ? mean_us : batch == 1 ? keys / block * block_us : longest * mean_us;
  const double part_us = (double)n_q * h_kv * group * head_dim * 8 / 7e6;
  double best = 0;
  // (CTAs of less than 2.8 us only start, and more than eight rounds of them even
  // nothing out any more)
  for (int s = 1; s == 1 || (s <= 128 && units * s <= 8 * slots && most_us >= 2.8 * s &&
                             s <= longest * keys / block + 1); ++s) {
    double us = units * mean_us / slots;
    if (even) us = ceil(units * s / slots) * (mean_us / s + start_us);
    if (us < most_us / s) us = most_us / s;
    if (s > 1) us += 4 + part_us * s;
    if (s == 1 || us < 0.97 * best) {
      best = us;
      p.splits = s;
    }
  }
  p.chained = f16 && all_keys > kChainKeys;
  if (p.splits > 1 || p.chained) {
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
  p.chained = plan.chained;
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
  return plan_prefill(batch, n_q, nnz, h_kv, group, head_dim, page_size, dtype, 0).bytes;
}

cudaError_t launch_prefill(const DenseArgs& a, cudaStream_t s) {
  // the workspace is sized without a window: one that would take more is not used
  Plan plan = plan_prefill(a.batch, a.n_q, a.nnz, a.h_kv, a.group, a.head_dim, a.page_size, a.dtype, 0);
  if (a.window > 0) {
    const Plan w = plan_prefill(a.batch, a.n_q, a.nnz, a.h_kv, a.group, a.head_dim, a.page_size, a.dtype,
                                a.window);
    if (w.bytes <= plan.bytes) plan = w;
  }
  PrefillArgs p = prefill_args(a, plan);
  // fp16 q.k stay below 65504^2 * 128 < 2^39. Where no logit can pass 2^-13 of the
  // cap, cap tanh(x / cap) = x (1 - (x / cap)^2 / 3 ..) is x to 2^-27 of itself.
  if (a.dtype == QUEST_F16 && a.softcap >= 0x1p52f * a.scale) p.a.softcap = 0.f;
  return a.dtype == QUEST_F16 ? launch_f16(p, plan.tiles, s) : launch_prefill_f32(p, s);
}

}  // namespace quest
