// Prompt attention: what the fp16 and the fp32 kernel share. Rows are cut into
// blocks of one request's tokens times the group's heads; with few blocks the
// keys of each are cut into equal parts, whose results are joined at the end.
#pragma once

#include "dense.cuh"
#include "tc.cuh"

namespace quest {

// A tensor-core accumulator is no fp32 sum: a product of 16 keys is added with each of
// its terms cut to a quarter of the accumulator's last place, and the result to one,
// towards zero. That takes 2.5 units of 2^-23 on average, half of it over a growing
// chain: 65536 keys left outputs 6e-4 short, more than their rounding to fp16. So a
// chain has at most this many keys (8e-5); then its sums go to the workspace in
// fp32. 16384 tokens of 32 heads take 1.30 ms with one chain of 16384, 1.34 with
// 8192 and 1.39 with 4096.
constexpr int kChainKeys = 8192;

struct PrefillArgs {
  DenseArgs a;
  int32_t blocks;          // row blocks, an upper bound (sum over requests)
  int32_t splits;          // equal parts of each block's keys
  int32_t near_heads;      // KV heads that run side by side
  int32_t chained;         // fp16: sums of more than kChainKeys keys go through part_o
  float* part_o;           // [splits, n_q, h_q, D]: chains' sums, then normalised parts
  float* part_lse;         // [splits, n_q, h_q]: chains' maxima, then parts' lse, base 2
  uint32_t wait_limit;

  // CTAs in order: groups of KV heads whose keys stay in L2 while all row
  // blocks pass (see the plan), row blocks (find_block's order), splits, heads.
  __device__ __forceinline__ void place(int cta, int h_kv, int* g, int* split, int* idx) const {
    const int full = blocks * splits * near_heads, group = cta / full;
    const int heads = min(near_heads, h_kv - group * near_heads), in = cta - group * full;
    *g = group * near_heads + in % heads;
    *split = in / heads % splits;
    *idx = in / heads / splits;
  }
};

// Finds row block `idx`, of blocks of `tokens` tokens: of up to 32 requests those
// whose rows start furthest in the cache first, else in their order; of a
// request the last rows, which see most keys, first. Long work so starts early
// and the device ends on short (16 requests of 2 to 32768 tokens, four rows
// each: 185 -> 168 us).
__device__ __forceinline__ bool find_block(const DenseArgs& a, int tokens, int idx, int lane,
                                           int* r_out, int* b_out) {
  auto rows_of = [&](int r) { return r < a.batch ? min(a.q_indptr[r + 1], a.n_q) - a.q_indptr[r] : 0; };
  auto blocks_of = [&](int n) { return n > 0 ? (n + tokens - 1) / tokens : 0; };
  // the lane whose request holds block `at` of its own
  auto found = [&](int r0, int at, int cnt) {
    const unsigned hit = __ballot_sync(FULL, at >= 0 && at < cnt);
    if (!hit) return false;
    *r_out = r0 + __ffs(hit) - 1;
    *b_out = __shfl_sync(FULL, cnt - 1 - at, __ffs(hit) - 1);
    return true;
  };
  if (a.batch <= 32) {
    const int n = rows_of(lane), cnt = blocks_of(n);
    const int from = lane < a.batch ? a.seq_lens[lane] - n : 0;
    int before = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const int ck = __shfl_sync(FULL, cnt, k), fk = __shfl_sync(FULL, from, k);
      before += fk > from || (fk == from && k < lane) ? ck : 0;
    }
    return found(0, idx - before, cnt);
  }
  int base = 0;
  for (int r0 = 0; r0 < a.batch; r0 += 128) {          // four loads in flight
    int cnt[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) cnt[k] = blocks_of(rows_of(r0 + 32 * k + lane));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int all = __reduce_add_sync(FULL, cnt[k]);
      if (idx < base + all) {
        int incl = cnt[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(FULL, incl, o);
          if (lane >= o) incl += t;
        }
        return found(r0 + 32 * k, idx - base - (incl - cnt[k]), cnt[k]);
      }
      base += all;
    }
  }
  return false;
}

// Joins the splits of each row by log-sum-exp. Few splits: a warp per (row,
// query head). Many (of few rows, then): a CTA of eight warps per (row, query
// head), each warp every eighth split, summed in shared memory in a fixed order.
constexpr int kJoinWarpSplits = 8;
template <typename O, int D, bool WIDE>
__global__ void __launch_bounds__(256) prefill_join_kernel(const PrefillArgs p) {
  constexpr int E = D / 32, NW = WIDE ? 8 : 1;         // warps of a row
  __shared__ float s_o[WIDE ? 8 : 1][WIDE ? D : 1], s_sum[8], s_m[8];
  const DenseArgs& a = p.a;
  const size_t all = (size_t)a.n_q * a.h_kv * a.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t at = WIDE ? blockIdx.x : (size_t)blockIdx.x * 8 + warp;
  if (at >= all || at >= (size_t)a.q_indptr[a.batch] * a.h_kv * a.group) return;
  // the row's maximum, then each split's weight in the lanes of its warp
  const int first = WIDE ? warp : 0;                   // this warp's splits: first, first + NW, ..
  float m = -INFINITY, sum = 0.f, o[E] = {};
  for (int s0 = first; s0 < p.splits; s0 += 32 * NW) {
    const int mine = s0 + lane * NW;
    const float lse = mine < p.splits ? p.part_lse[mine * all + at] : -INFINITY;
    const float mx = fmaxf(m, warp_max(lse));
    if (mx == -INFINITY) continue;
    const float f = ex2(m - mx), w = ex2(lse - mx);
    m = mx;
    sum = sum * f + warp_sum(w);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f;
    const int n = min(32, (p.splits - s0 + NW - 1) / NW);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float* src = p.part_o + ((size_t)(s0 + k * NW) * all + at) * D + lane * E;
      const float ws = __shfl_sync(FULL, w, k);
      float v[E];
      if constexpr (E == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
      else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(ws, v[e], o[e]);
    }
  }
  if constexpr (WIDE) {
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
    if (lane == 0) {
      s_sum[warp] = sum;
      s_m[warp] = m;
    }
    __syncthreads();
    if (warp > 0) return;
    for (int w = 0; w < 8; ++w) m = fmaxf(m, s_m[w]);
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int w = 0; w < 8; ++w) {
      const float f = s_m[w] == -INFINITY ? 0.f : ex2(s_m[w] - m);
      sum = fmaf(f, s_sum[w], sum);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(f, s_o[w][lane * E + e], o[e]);
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  O* dst = static_cast<O*>(a.out) + at * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    if constexpr (sizeof(O) == 2)
      *reinterpret_cast<__half2*>(dst + e) = __floats2half2_rn(o[e] * inv, o[e + 1] * inv);
    else
      *reinterpret_cast<float2*>(dst + e) = make_float2(o[e] * inv, o[e + 1] * inv);
  }
  if (lane == 0 && a.lse) a.lse[at] = sum > 0.f ? (m + lg2(sum)) * LN2 : -INFINITY;
}

template <typename O, int D> cudaError_t launch_prefill_join(const PrefillArgs& p, cudaStream_t s) {
  const size_t rows = (size_t)p.a.n_q * p.a.h_kv * p.a.group;
  if (p.splits > kJoinWarpSplits) prefill_join_kernel<O, D, true><<<(unsigned)rows, 256, 0, s>>>(p);
  else prefill_join_kernel<O, D, false><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace quest
