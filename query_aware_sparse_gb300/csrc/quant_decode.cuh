// Decode attention over the E4M3 cache: one query per request over the pages
// that a list or the page table names.
//
// Mathematics. A stored value is code * 2^e, an fp16 number. The products run
// on mma.sync m16n8k16 in fp16: the codes of K as they are (exact), 2^e of a
// token as a factor of its logit; the codes of V times 2^e (exact), since the
// weights would leave fp16's range with it. The running softmax is
// dense_decode.cuh's (WarpMma): against the stored values, the output is as accurate
// as it says there.
//
// Bound: HBM, 2 (D + 1) bytes a token and KV head, half of an fp16 cache; small
// calls the chain launch - lengths - page ids - pages - join.
//
// Two splits, chosen on the host (quant_decode.cu): the equal runs and the join
// kernel of dense_decode.cuh, with a page of one KV head (its record, one bulk
// copy) as the tile; and a cluster per unit below, which starts and joins in one
// launch. A third, runs whose last CTA joins them behind a counter, took 17.1
// instead of 11.3 us for 32 heads of 128 pages: barriers, a fence and an atomic
// in front of the same loads, by code that is cold.
//
// Measured: 16 requests of 8192 to 131072 tokens, 8 KV heads of 4 (128 dims),
// 337 to 344 us, 6820 to 6680 GB/s (98% of the copy rate and more); 256 pages of each 25 us (72%); 128 of
// 2048 pages of 32 heads 7.7 us; 1000 tokens of one head 4.1 us.
#pragma once

#include "dense_decode.cuh"
#include "e4m3_page.cuh"

namespace quest {

struct PageRecords { const uint8_t* pool; };

template <int D, int S> struct RecordShape {
  static constexpr int TT = S;
  static constexpr uint32_t STAGE = 2 * S * (D + 1);
  static constexpr int WARPS = D == 64 ? 16 : 12;
  static constexpr int STAGES = 200704 / WARPS / STAGE;
  static constexpr uint32_t SMEM = 1024 + WARPS * STAGES * STAGE;
  static_assert(STAGE % 16 == 0 && STAGES >= 2 && STAGES <= 32, "bulk copies of 16-byte pieces");
};

// Lane (g, t) = (lane / 4, lane % 4) reads 16 bytes at a time: 16 dims of K of
// tokens g and g + 8 (dims 64 j + 16 t + ..), or V of four dims (32 i + 4 g + ..)
// and tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9.
//
// The two groups of 16 tokens of a 32-token page go through together, so that
// one's chain of loads, products and shuffles hides the other's. PACK (up to
// four heads): the heads stand in the MMA's columns twice. The first group's
// logits are taken from columns 0..3 and the second's from 4..7, one softmax
// step serves both, and the two halves of a weight meet a group's values in one
// product, in a column each. What a head's two columns hold adds up at the end.
// (64 dims, 63 requests of up to 8192 tokens, capped: 24.2 us without; 16000
// tokens of one head 15.4 -> 11.7. Two pages of 16 tokens together gained nothing.)
template <int D, int S, bool PACK> struct WarpE4M3 : WarpMma<D> {
  using Base = WarpMma<D>;
  using Shape = RecordShape<D, S>;
  using Source = PageRecords;
  using Base::acc;
  using Base::l;
  using Base::m;
  using Base::qb;
  using Base::sum;
  static constexpr bool kQueryShared = false;

  __device__ __forceinline__ static void copy(const Source& src, const DenseArgs& a, int id, int g, int,
                                              uint32_t dst, uint64_t* bar, uint64_t pol) {
    const uint8_t* rec = src.pool + ((size_t)id * a.h_kv + g) * Shape::STAGE;
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
        :: "r"(dst), "l"(rec), "r"(Shape::STAGE), "r"(smem_u32(bar)), "l"(pol) : "memory");
  }

  __device__ __forceinline__ void begin(const DenseArgs& a, int r, int g, int lane, float*) {
    const int t = lane & 3, head = PACK ? lane >> 2 & 3 : lane >> 2;
    const __half* q = static_cast<const __half*>(a.q) + (((size_t)r * a.h_kv + g) * a.group + head) * D;
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint2 v = make_uint2(0u, 0u);
        if (head < a.group) v = *reinterpret_cast<const uint2*>(q + 64 * j + 16 * t + 4 * w);
        qb[4 * j + w][0] = v.x;
        qb[4 * j + w][1] = v.y;
      }
    Base::clear(a, g, PACK ? lane & ~2 : lane);        // columns 4.. take the slopes of 0..
  }

  __device__ __forceinline__ static uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
  }
  __device__ __forceinline__ static uint32_t lds1(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
  }
  // Scales of tokens at, at + 1, as fp16.
  __device__ __forceinline__ static uint32_t scale_pair(uint32_t at) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
    return scale_h2(__byte_perm(v, 0u, 0x4140));
  }

  // Products of the heads with the codes of 16 tokens' keys.
  __device__ __forceinline__ void products(uint32_t rec, int sub, int lane, float (&s)[4]) const {
    const uint32_t k_s = rec + (16 * sub + (lane >> 2)) * 64 + 16 * (lane & 3);
    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const uint4 x = lds16(k_s + j * S * 64), y = lds16(k_s + j * S * 64 + 512);
      const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t a0 = e4m3_pair(xw[w]), a2 = e4m3_pair(xw[w] >> 16);
        const uint32_t a1 = e4m3_pair(yw[w]), a3 = e4m3_pair(yw[w] >> 16);
        const int k = 4 * j + w;
        if (w & 1) mma_f16_16816(s1, a0, a1, a2, a3, qb[k][0], qb[k][1]);
        else mma_f16_16816(s0, a0, a1, a2, a3, qb[k][0], qb[k][1]);
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) s[c] = s0[c] + s1[c];
  }
  // What a token's value is multiplied by, and which of four tokens' bytes are
  // there: slots without a token may hold anything, so they are cleared.
  struct Values { uint32_t u0, u1, there; };
  __device__ __forceinline__ static Values values(uint32_t rec, int sub, int tok, int held, int lane) {
    const int t = lane & 3;
    const uint32_t at = rec + 2 * S * D + S + 16 * sub + 2 * t;
    Values v{scale_pair(at), scale_pair(at + 8), 0xffffffffu};
    if (tok + 16 > held) {
      const int n = held - tok;
      v.there = (2 * t < n ? 0xffu : 0u) | (2 * t + 1 < n ? 0xff00u : 0u) | (2 * t + 8 < n ? 0xff0000u : 0u) |
                (2 * t + 9 < n ? 0xff000000u : 0u);
      v.u0 &= __byte_perm(v.there, 0u, 0x1100);
      v.u1 &= __byte_perm(v.there, 0u, 0x3322);
    }
    return v;
  }
  // acc += V^T P^T of 16 tokens and 32 dims, for N columns' halves of weights.
  template <int N>
  __device__ __forceinline__ void add(uint32_t rec, int sub, int i, int lane, const Values& v, const uint32_t (&w)[N][2]) {
    const uint4 x = lds16(rec + S * D + sub * D * 16 + i * 512 + lane * 16);
    const uint32_t xw[4] = {x.x & v.there, x.y & v.there, x.z & v.there, x.w & v.there};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a0 = mul_h2(e4m3_pair(xw[2 * h]), v.u0), a2 = mul_h2(e4m3_pair(xw[2 * h] >> 16), v.u1);
      const uint32_t a1 = mul_h2(e4m3_pair(xw[2 * h + 1]), v.u0), a3 = mul_h2(e4m3_pair(xw[2 * h + 1] >> 16), v.u1);
#pragma unroll
      for (int n = 0; n < N; ++n) mma_f16_16816(acc[2 * i + h], a0, a1, a2, a3, w[n][0], w[n][1]);
    }
  }

  // Tokens tok0 .. + 15 at (rec0, sub0) of shared memory and, with `two`, tok1
  // .. + 15 at (rec1, sub1).
  __device__ __forceinline__ void pair(const DenseArgs& a, const Request& rq, int tok0, uint32_t rec0, int sub0,
                                       bool two, int tok1, uint32_t rec1, int sub1, float scale2, int lane) {
    const int g = lane >> 2;
    float s0[4], s1[4] = {0.f, 0.f, 0.f, 0.f};
    products(rec0, sub0, lane, s0);
    if (two) products(rec1, sub1, lane, s1);
    const Values v0 = values(rec0, sub0, tok0, rq.held, lane);
    Values v1{};
    if (two) v1 = values(rec1, sub1, tok1, rq.held, lane);
    if constexpr (PACK) {
      const bool second = lane & 2;
      const uint32_t scales = (second && two ? rec1 + 16 * sub1 : rec0 + 16 * sub0) + 2 * S * D + g;
      const float fa = scale_f(lds1(scales)), fb = scale_f(lds1(scales + 8));
      const float s[4] = {(second ? s1[0] : s0[0]) * fa, (second ? s1[1] : s0[1]) * fa,
                          (second ? s1[2] : s0[2]) * fb, (second ? s1[3] : s0[3]) * fb};
      uint32_t hi[2], lo[2], w0[1][2], w1[1][2];
      // without a second group its columns see nothing
      Base::template weigh<true>(a, rq, second ? (two ? tok1 : rq.hi) : tok0, [&](int c) { return s[c]; }, scale2, lane, hi, lo);
#pragma unroll
      for (int i = 0; i < 2; ++i) {                    // a group's lower halves to the other columns
        const uint32_t away = __shfl_xor_sync(FULL, lo[i], 16);
        w0[0][i] = g < 4 ? hi[i] : away;
        w1[0][i] = g < 4 ? away : hi[i];
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        add<1>(rec0, sub0, i, lane, v0, w0);
        if (two) add<1>(rec1, sub1, i, lane, v1, w1);
      }
    } else {
      auto scaled = [&](uint32_t rec, int sub, float (&s)[4]) {
        const uint32_t scales = rec + 2 * S * D + 16 * sub + g;
        const float fa = scale_f(lds1(scales)), fb = scale_f(lds1(scales + 8));
        s[0] *= fa; s[1] *= fa; s[2] *= fb; s[3] *= fb;
      };
      uint32_t w0[2][2], w1[2][2];
      scaled(rec0, sub0, s0);
      if (two) scaled(rec1, sub1, s1);
      Base::weigh(a, rq, tok0, [&](int c) { return s0[c]; }, scale2, lane, w0[0], w0[1]);
      if (two) {
        // a new maximum rescales sums that the first group's products are not
        // in yet: its weights are rescaled with them
        const float m0 = m[0], m1 = m[1];
        Base::weigh(a, rq, tok1, [&](int c) { return s1[c]; }, scale2, lane, w1[0], w1[1]);
        if (__any_sync(FULL, m[0] != m0 || m[1] != m1)) Base::reweigh(m0, m1, lane, w0[0], w0[1]);
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        add<2>(rec0, sub0, i, lane, v0, w0);
        if (two) add<2>(rec1, sub1, i, lane, v1, w1);
      }
    }
    if ((Base::since += two ? 2 : 1) >= 8) Base::settle();
  }

  // the page of tokens tok0 .. tok0 + S - 1 in shared memory at rec
  __device__ __forceinline__ void tile(const DenseArgs& a, const Request& rq, int tok0, uint32_t rec,
                                       const float*, float scale2, int lane) {
    if constexpr (S == 16) {
      pair(a, rq, tok0, rec, 0, false, 0, rec, 0, scale2, lane);
    } else {
      const bool first = tok0 < rq.hi && tok0 + 16 > rq.lo, second = tok0 + 16 < rq.hi && tok0 + 32 > rq.lo;
      if (first && second) pair(a, rq, tok0, rec, 0, true, tok0 + 16, rec, 1, scale2, lane);
      else if (first) pair(a, rq, tok0, rec, 0, false, 0, rec, 0, scale2, lane);
      else if (second) pair(a, rq, tok0 + 16, rec, 1, false, 0, rec, 0, scale2, lane);
    }
  }

  template <typename F>
  __device__ __forceinline__ void finish(const DenseArgs& a, bool whole, int lane, F put) {
    if constexpr (PACK) {                              // a head's two columns
      Base::settle();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[c] += __shfl_xor_sync(FULL, l[c], 2);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          sum[k][c] += __shfl_xor_sync(FULL, sum[k][c], 2);
          sum[k][2 + c] += __shfl_xor_sync(FULL, sum[k][2 + c], 2);
        }
      }
    }
    Base::finish_heads(a, whole, lane, put, [&](float* o, int c, float f) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        *reinterpret_cast<float4*>(o + 32 * i + 4 * (lane >> 2)) =
            make_float4(sum[2 * i][c] * f, sum[2 * i][2 + c] * f, sum[2 * i + 1][c] * f, sum[2 * i + 1][2 + c] * f);
    });
  }
};

// ---------------------------------------------------------------------------
// Few tiles: a cluster of up to eight CTAs of four warps takes one unit, its
// parts meet in distributed shared memory, and one launch is all there is.
// ---------------------------------------------------------------------------
constexpr int kUnitWarps = 4, kUnitCtasPerSm = 3;

template <int D, int S> struct UnitShape {
  static constexpr uint32_t STAGE = RecordShape<D, S>::STAGE;
  static constexpr int STAGES = 66560 / kUnitWarps / STAGE;
  static constexpr uint32_t RING = STAGES * STAGE, SMEM = kUnitWarps * RING;
  static_assert(STAGES <= 32 && kUnitCtasPerSm * (SMEM + 3072) <= 227 * 1024, "three CTAs per SM");
  // a part (o and m, l of up to eight heads) behind a part, in a ring that is through
  static constexpr uint32_t PART = 8 * D * 4 + 8 * 8;
  static_assert(2 * PART <= RING && PART % 16 == 0, "parts use the rings");
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t in_cta(uint32_t at, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at));
  return v;
}

// Joins N parts' four dims: m, l and o of part i from ml(i) and o(i).
template <int N, typename M, typename O>
__device__ __forceinline__ void join_four(int n, M ml, O o, float& m, float& l, float4& sum) {
  float2 x[N];
  float4 v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = make_float2(-INFINITY, 0.f);
    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n) { x[i] = ml(i); v[i] = o(i); }
  }
  m = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, x[i].x);
  l = 0.f;
  sum = make_float4(0.f, 0.f, 0.f, 0.f);
  if (m == -INFINITY) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float f = ex2(x[i].x - m);
    l = fmaf(f, x[i].y, l);
    sum.x = fmaf(f, v[i].x, sum.x);
    sum.y = fmaf(f, v[i].y, sum.y);
    sum.z = fmaf(f, v[i].z, sum.z);
    sum.w = fmaf(f, v[i].w, sum.w);
  }
}

// LIST as in dense_decode_kernel. Grid: a cluster, of any size up to 8, per unit.
template <int D, int S, bool LIST, bool PACK>
__global__ void __launch_bounds__(kUnitWarps * 32, kUnitCtasPerSm)
quant_unit_kernel(const PageRecords source, const DecodeArgs p) {
  using W = WarpE4M3<D, S, PACK>;
  using Sh = UnitShape<D, S>;
  constexpr int NST = Sh::STAGES;
  extern __shared__ __align__(128) uint8_t unit_smem[];
  __shared__ __align__(8) uint64_t s_bar[kUnitWarps][NST];
  __shared__ int s_tok[kUnitWarps][NST];
  const DenseArgs& a = p.a;
  const int G = a.group, warp = __shfl_sync(FULL, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  int ctas;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
  const int unit = blockIdx.x / ctas, r = unit / a.h_kv, g = unit % a.h_kv;
  const uint32_t smem = smem_u32(unit_smem), ring = smem + warp * Sh::RING;
  if (lane < NST) mbar_init(&s_bar[warp][lane], 1);
  fence_mbar_init();
  __syncwarp();
  pdl_wait();
  pdl_launch_dependents();

  // The warp's tiles: every (4 ctas)-th of the unit's, 32 of them looked up at
  // a time, one per lane; those without a page or a token are left out there.
  const int step = kUnitWarps * ctas, own = rank * kUnitWarps + warp;
  int at = own, pages = -1, ids = -1;
  const size_t list = (size_t)unit * p.sel_k;
  if (LIST && at + lane * step < p.sel_k) {            // on the way beside the length
    pages = p.sel_logical[list + at + lane * step];
    ids = p.sel_phys[list + at + lane * step];
  }
  W w;
  w.begin(a, r, g, lane, nullptr);
  unsigned* err = own == 0 && g == 0 ? a.err : nullptr;
  const Request rq = LIST ? listed_request(p, r) : request_of<S>(a, r, err);
  unsigned left = 0;
  auto look_up = [&](bool first) {
    const int i = at + lane * step;
    at += 32 * step;
    if constexpr (LIST) {
      if (!first) {
        pages = i < rq.tiles ? p.sel_logical[list + i] : -1;
        ids = i < rq.tiles ? p.sel_phys[list + i] : -1;
      }
      if (pages >= (rq.held + S - 1) / S) {            // no token of the request
        report(a.err, QUEST_DEVERR_EMPTY_PAGE);
        pages = -1;
      }
    } else {
      pages = i < rq.tiles ? rq.tile0 + i : -1;
      ids = i < rq.tiles ? a.page_indices[rq.e0 + rq.tile0 + i] : -1;
    }
    if (pages >= 0 && (ids < 0 || ids >= a.n_phys)) {
      report(a.err, QUEST_DEVERR_PAGE_RANGE);
      pages = -1;
    }
    left = __ballot_sync(FULL, pages >= 0);
  };
  look_up(true);

  const uint64_t pol = evict_first_policy();
  const bool fault = a.test_fault == 2 && blockIdx.x == 0 && warp == 0;
  int issued = 0;
  auto issue = [&] {                                   // the next tile into the ring
    while (!left && at < rq.tiles) look_up(false);
    if (!left) return;
    const int src = __ffs(left) - 1, st = issued % NST;
    left &= left - 1;
    const int id = __shfl_sync(FULL, ids, src), lp = __shfl_sync(FULL, pages, src);
    if (lane == 0) {
      s_tok[warp][st] = lp * S;
      mbar_expect_tx(&s_bar[warp][st], Sh::STAGE + (fault && issued == 0 ? 16 : 0));
      W::copy(source, a, id, g, 0, ring + st * Sh::STAGE, &s_bar[warp][st], pol);
    }
    ++issued;
  };
  for (int k = 0; k < NST; ++k) issue();
  const float scale2 = a.scale * LOG2E;
  int done = 0, st = 0;
  uint32_t phase = 0;
  for (; done < issued; ++done) {
    __syncwarp();
    if (!warp_wait_bounded(&s_bar[warp][st], phase >> st & 1, p.wait_limit)) break;
    phase ^= 1u << st;
    w.tile(a, rq, s_tok[warp][st], ring + st * Sh::STAGE, nullptr, scale2, lane);
    __syncwarp();
    issue();
    if (++st == NST) st = 0;
  }
  if (done < issued) {                                 // report, and wait for the copies in flight
    if (lane == 0) report(a.err, QUEST_DEVERR_WAIT_TIMEOUT);
    for (int k = done; k < issued; ++k, st = st + 1 == NST ? 0 : st + 1)
      warp_wait_bounded(&s_bar[warp][st], phase >> st & 1, p.wait_limit);
  }

  auto meet = [] {                                     // every CTA of the cluster, whole warps
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  };
  // the warp's part into its ring, the CTA's behind the first warp's
  auto o_at = [&](uint32_t part, int h) { return part + h * D * 4; };
  auto ml_at = [&](uint32_t part, int h) { return part + G * D * 4 + h * 8; };
  w.finish(a, false, lane, [&](int h, float m, float l, bool mine) {
    float* o = reinterpret_cast<float*>(unit_smem + warp * Sh::RING);
    if (mine) *reinterpret_cast<float2*>(o + G * D + 2 * h) = make_float2(m, l);
    return o + h * D;
  });
  __syncthreads();
  const size_t row = (size_t)unit * G;
  auto put = [&](int h, int d4, float m, float l, float4 o) {
    const float f = l > 0.f ? 1.f / l : 0.f;
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + (row + h) * D + d4 * 4) =
        make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    if (d4 == 0 && a.lse) a.lse[row + h] = l > 0.f ? (m - 6.f + lg2(l)) * LN2 : -INFINITY;
  };
  const int items = G * (D / 4);
  const uint32_t cta_part = smem + Sh::PART;
  for (int i = threadIdx.x; i < items; i += kUnitWarps * 32) {
    const int h = i / (D / 4), d4 = i % (D / 4);
    float m, l;
    float4 o;
    join_four<kUnitWarps>(kUnitWarps, [&](int k) { return ld_cluster2(in_cta(ml_at(smem + k * Sh::RING, h), rank)); },
                          [&](int k) { return ld_cluster4(in_cta(o_at(smem + k * Sh::RING, h) + d4 * 16, rank)); }, m, l, o);
    if (ctas == 1) {
      put(h, d4, m, l, o);
    } else {
      float* to = reinterpret_cast<float*>(unit_smem + Sh::PART);
      *reinterpret_cast<float4*>(to + h * D + d4 * 4) = o;
      if (d4 == 0) *reinterpret_cast<float2*>(to + G * D + 2 * h) = make_float2(m, l);
    }
  }
  if (ctas == 1) return;
  meet();
  for (int i = rank * kUnitWarps * 32 + threadIdx.x; i < items; i += ctas * kUnitWarps * 32) {
    const int h = i / (D / 4), d4 = i % (D / 4);
    float m, l;
    float4 o;
    join_four<8>(ctas, [&](int k) { return ld_cluster2(in_cta(ml_at(cta_part, h), k)); },
                 [&](int k) { return ld_cluster4(in_cta(o_at(cta_part, h) + d4 * 16, k)); }, m, l, o);
    put(h, d4, m, l, o);
  }
  // a CTA's part stays until every other has read it
  meet();
}

}  // namespace quest
