// Decode attention over the E4M3 cache: one query per request over the pages
// that a list or the page table names. The split over warps, the ring and the
// join are dense_decode.cuh's; here a tile is a page of one KV head, its record
// (e4m3_page.cuh) one bulk copy.
//
// Mathematics. A stored value is code * 2^e, an fp16 number. The products run
// on mma.sync m16n8k16 in fp16: the codes of K as they are (exact), 2^e of a
// token as a factor of its logit; the codes of V times 2^e (exact), since the
// weights would leave fp16's range with it. Everything else is as for fp16 keys,
// so the output keeps fp32 accuracy against the stored values.
//
// Bound: HBM, 2 (D + 1) bytes a token and KV head, half of an fp16 cache.
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
template <int D, int S> struct WarpE4M3 : WarpMma<D> {
  using Base = WarpMma<D>;
  using Shape = RecordShape<D, S>;
  using Source = PageRecords;
  using Base::acc;
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
    const int t = lane & 3;
    const __half* q = Base::query(a, r, g, lane);
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint2 v = make_uint2(0u, 0u);
        if (q) v = *reinterpret_cast<const uint2*>(q + 64 * j + 16 * t + 4 * w);
        qb[4 * j + w][0] = v.x;
        qb[4 * j + w][1] = v.y;
      }
    Base::clear(a, g, lane);
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

  // the page of tokens tok0 .. tok0 + S - 1 in shared memory at rec
  __device__ __forceinline__ void tile(const DenseArgs& a, const Request& rq, int tok0, uint32_t rec,
                                       const float*, float scale2, int lane) {
#pragma unroll
    for (int sub = 0; sub < S / 16; ++sub) {
      const int tok = tok0 + 16 * sub;
      if (tok >= rq.hi || tok + 16 <= rq.lo) continue;
      rows(a, rq, tok, rec, sub, scale2, lane);
    }
  }

  __device__ __forceinline__ void rows(const DenseArgs& a, const Request& rq, int tok, uint32_t rec, int sub,
                                       float scale2, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const uint32_t k_s = rec + (16 * sub + g) * 64 + 16 * t, v_s = rec + S * D + (sub * D * 16 + lane * 16);
    const uint32_t scales = rec + 2 * S * D + 16 * sub;
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
    const float fa = scale_f(lds1(scales + g)), fb = scale_f(lds1(scales + g + 8));
    const float s[4] = {(s0[0] + s1[0]) * fa, (s0[1] + s1[1]) * fa, (s0[2] + s1[2]) * fb, (s0[3] + s1[3]) * fb};
    uint32_t hi[2], lo[2];
    Base::weigh(a, rq, tok, s, scale2, lane, hi, lo);
    uint32_t u0 = scale_pair(scales + S + 2 * t), u1 = scale_pair(scales + S + 2 * t + 8);
    // slots without a token may hold anything: their codes and scales are cleared
    uint32_t there = 0xffffffffu;
    if (tok + 16 > rq.held) {
      const int n = rq.held - tok;
      there = (2 * t < n ? 0xffu : 0u) | (2 * t + 1 < n ? 0xff00u : 0u) | (2 * t + 8 < n ? 0xff0000u : 0u) |
              (2 * t + 9 < n ? 0xff000000u : 0u);
      u0 &= __byte_perm(there, 0u, 0x1100);
      u1 &= __byte_perm(there, 0u, 0x3322);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 x = lds16(v_s + i * 512);
      const uint32_t xw[4] = {x.x & there, x.y & there, x.z & there, x.w & there};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t a0 = mul_h2(e4m3_pair(xw[2 * h]), u0), a2 = mul_h2(e4m3_pair(xw[2 * h] >> 16), u1);
        const uint32_t a1 = mul_h2(e4m3_pair(xw[2 * h + 1]), u0), a3 = mul_h2(e4m3_pair(xw[2 * h + 1] >> 16), u1);
        mma_f16_16816(acc[2 * i + h], a0, a1, a2, a3, hi[0], hi[1]);
        mma_f16_16816(acc[2 * i + h], a0, a1, a2, a3, lo[0], lo[1]);
      }
    }
    if (++Base::since == 8) Base::settle();
  }

  template <typename F>
  __device__ __forceinline__ void finish(const DenseArgs& a, bool whole, int lane, F put) {
    Base::finish_heads(a, whole, lane, put, [&](float* o, int c, float f) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        *reinterpret_cast<float4*>(o + 32 * i + 4 * (lane >> 2)) =
            make_float4(sum[2 * i][c] * f, sum[2 * i][2 + c] * f, sum[2 * i + 1][c] * f, sum[2 * i + 1][2 + c] * f);
    });
  }
};

}  // namespace quest
