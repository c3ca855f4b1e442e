// Device parts of the appends that treat queries and keys on the way
// (rope_append.cu, norm_append.cu): the touched pages, angles, the rotation of
// a lane's pairs, and page summaries.
#pragma once

#include "common.cuh"
#include "dense.h"

namespace quest {

constexpr int kMaxPage = 32;      // tokens per page, at most

// Pages of request r that the call touches.
__device__ __forceinline__ int touched(const RopeAppendArgs& a, int r) {
  if (r >= a.batch) return 0;
  const int n = a.append_indptr[r + 1] - a.append_indptr[r], p0 = a.seq_lens_before[r];
  return n > 0 && p0 >= 0 ? (p0 + n - 1) / a.page_size - p0 / a.page_size + 1 : 0;
}
__device__ __forceinline__ int warp_running_sum(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(FULL, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// The `seg`-th (request, touched page) of the call, counted in request order;
// false past the last one. Up to 32 requests every warp looks by itself, else
// the CTA scans as many as it has threads at a time.
template <int NT>
__device__ bool touched_page(const RopeAppendArgs& a, int seg, int* r_out, int* j_out) {
  __shared__ int s_r, s_j, s_sum[NT / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (a.batch <= 32) {
    const int pages = touched(a, lane), at = seg - (warp_running_sum(pages, lane) - pages);
    const unsigned hit = __ballot_sync(FULL, at >= 0 && at < pages);
    if (!hit) return false;
    *r_out = __ffs(hit) - 1;
    *j_out = __shfl_sync(FULL, at, __ffs(hit) - 1);
    return true;
  }
  int base = 0;
  if (threadIdx.x == 0) s_r = -1;
  for (int r0 = 0; r0 < a.batch; r0 += NT) {
    const int pages = touched(a, r0 + (int)threadIdx.x), incl = warp_running_sum(pages, lane);
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int before = base + incl - pages;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) before += s_sum[w];
      base += s_sum[w];
    }
    const int at = seg - before;
    if (at >= 0 && at < pages) { s_r = r0 + (int)threadIdx.x; s_j = at; }
    __syncthreads();
    if (s_r >= 0) break;
  }
  *r_out = s_r;
  *j_out = s_j;
  return s_r >= 0;
}

// Radians per position -> turns per position as a 64-bit fraction, modulo one
// turn: the double's mantissa times 2^64 / (2 pi), shifted by its exponent. In
// integers: the few fp64 units would take longer than everything else here.
__device__ __forceinline__ unsigned long long turn_fraction(double inv_freq) {
  const unsigned long long bits = (unsigned long long)__double_as_longlong(inv_freq);
  const int e = (int)(bits >> 52 & 0x7ff) - 1023;
  const unsigned long long m = (bits << 11 | 1ull << 63) & (e > -1023 ? ~0ull : 0ull);
  const unsigned long long c = 2935890503282001226ull;         // 2^64 / (2 pi)
  const unsigned long long hi = __umul64hi(m, c), lo = m * c;
  const int s = 63 - e;                                        // (hi : lo) >> s, the low 64 bits
  unsigned long long f = 0;
  if (s >= 64) f = s < 128 ? hi >> (s - 64) : 0ull;
  else if (s > 0) f = hi << (64 - s) | lo >> s;
  else if (s > -64) f = lo << -s;
  return inv_freq < 0 ? 0ull - f : f;
}

template <typename T> struct Pack;
template <> struct Pack<__half> {
  __device__ __forceinline__ static uint32_t word(const float* x) {
    const __half2 h = __floats2half2_rn(x[0], x[1]);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ __forceinline__ static uint4 pack(const float* x) {
    return make_uint4(word(x), word(x + 2), word(x + 4), word(x + 6));
  }
};
template <> struct Pack<float> {
  __device__ __forceinline__ static uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};

// Rotate the VEC pairs held by two 16-byte vectors: pair e is (a[e], b[e]),
// or with IL the neighbours (2e, 2e + 1) of the two vectors in a row.
template <typename T, bool IL>
__device__ __forceinline__ void rotate(uint4& a, uint4& b, const float* cs, const float* sn) {
  constexpr int VEC = Elem<T>::kVec;
  float x[2 * VEC], y[2 * VEC], c[VEC], s[VEC];
  unpack16<T>(a, x);
  unpack16<T>(b, x + VEC);
#pragma unroll
  for (int e = 0; e < VEC; e += 4) {
    *reinterpret_cast<float4*>(c + e) = *reinterpret_cast<const float4*>(cs + e);
    *reinterpret_cast<float4*>(s + e) = *reinterpret_cast<const float4*>(sn + e);
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const int i = IL ? 2 * e : e, j = IL ? 2 * e + 1 : e + VEC;
    y[i] = x[i] * c[e] - x[j] * s[e];
    y[j] = x[j] * c[e] + x[i] * s[e];
  }
  a = Pack<T>::pack(y);
  b = Pack<T>::pack(y + VEC);
}

// Stored min/max of one 16-byte piece of dims as order-preserving keys, and
// back (E4M3 codes decode exactly to fp16 and are rounded outward again).
template <typename T, bool F8>
struct Box {
  using K = KeyOps<T>;
  uint4 mn, mx;
  __device__ __forceinline__ void clear() {
    mn = make_uint4(K::kMinInit, K::kMinInit, K::kMinInit, K::kMinInit);
    mx = make_uint4(K::kMaxInit, K::kMaxInit, K::kMaxInit, K::kMaxInit);
  }
  __device__ __forceinline__ static uint4 keys(uint4 v) {
    return make_uint4(K::to_key(v.x), K::to_key(v.y), K::to_key(v.z), K::to_key(v.w));
  }
  __device__ __forceinline__ static uint4 values(uint4 k) {
    return make_uint4(K::from_key(k.x), K::from_key(k.y), K::from_key(k.z), K::from_key(k.w));
  }
  __device__ __forceinline__ static uint4 decode(uint2 c) {
    return make_uint4(e4m3x4_lo_h2(c.x), e4m3x4_hi_h2(c.x), e4m3x4_lo_h2(c.y), e4m3x4_hi_h2(c.y));
  }
  __device__ __forceinline__ void load(const void* lo, const void* hi) {
    if constexpr (F8) {
      mn = keys(decode(*reinterpret_cast<const uint2*>(lo)));
      mx = keys(decode(*reinterpret_cast<const uint2*>(hi)));
    } else {
      mn = keys(ld_v4(lo));
      mx = keys(ld_v4(hi));
    }
  }
  __device__ __forceinline__ void fold(uint4 v) {
    const uint4 k = keys(v);
    join(k, k);
  }
  __device__ __forceinline__ static uint4 other(uint4 v, int o) {
    return make_uint4(__shfl_xor_sync(FULL, v.x, o), __shfl_xor_sync(FULL, v.y, o),
                      __shfl_xor_sync(FULL, v.z, o), __shfl_xor_sync(FULL, v.w, o));
  }
  __device__ __forceinline__ void join(int o) { join(other(mn, o), other(mx, o)); }
  __device__ __forceinline__ void join(uint4 lo, uint4 hi) {
    mn = make_uint4(K::kmin(mn.x, lo.x), K::kmin(mn.y, lo.y), K::kmin(mn.z, lo.z), K::kmin(mn.w, lo.w));
    mx = make_uint4(K::kmax(mx.x, hi.x), K::kmax(mx.y, hi.y), K::kmax(mx.z, hi.z), K::kmax(mx.w, hi.w));
  }
  __device__ __forceinline__ void store(void* lo, void* hi, bool& ovf) const {
    const uint4 a = values(mn), b = values(mx);
    if constexpr (F8) {
      *reinterpret_cast<uint2*>(lo) =
          make_uint2(e4m3x4_floor_h(a.x, a.y, ovf), e4m3x4_floor_h(a.z, a.w, ovf));
      *reinterpret_cast<uint2*>(hi) =
          make_uint2(e4m3x4_ceil_h(b.x, b.y, ovf), e4m3x4_ceil_h(b.z, b.w, ovf));
    } else {
      st_v4(lo, a);
      st_v4(hi, b);
    }
  }
};

// A lane's two pieces of a row, at tokens tg, tg + TG, ...: the loads of four
// tokens are in flight before the first is used, then `each` handles them and
// they are stored.
template <typename T, int TG, typename F>
__device__ __forceinline__ void walk_rows(const T* src, int64_t src_stride, T* dst, int64_t dst_stride,
                                     int da, int db, int tg, int ntok, F each) {
  constexpr int U = 4;
  for (int t0 = tg; t0 < ntok; t0 += U * TG) {
    uint4 x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t0 + u * TG < ntok) {
        x[u] = ld_v4(src + (t0 + u * TG) * src_stride + da);
        y[u] = ld_v4(src + (t0 + u * TG) * src_stride + db);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t0 + u * TG < ntok) {
        each(x[u], y[u], t0 + u * TG);
        st_v4(dst + (t0 + u * TG) * dst_stride + da, x[u]);
        st_v4(dst + (t0 + u * TG) * dst_stride + db, y[u]);
      }
  }
}

// CTAs of an append: (request, touched page) by KV heads; sets heads_per_cta.
// A request with n new tokens touches at most ceil(n / S) + 1 pages, each with
// one token at least. Few pages: the KV heads of one are spread over CTAs until
// there are `wanted`.
inline dim3 append_grid(RopeAppendArgs& a, long long wanted) {
  long long segs = (long long)(a.n_new + a.page_size - 1) / a.page_size + 2LL * a.batch;
  if (segs > a.n_new) segs = a.n_new;
  a.heads_per_cta = a.h_kv;
  while (a.heads_per_cta > 1 && segs * ((a.h_kv + a.heads_per_cta - 1) / a.heads_per_cta) < wanted)
    a.heads_per_cta = (a.heads_per_cta + 1) / 2;
  return dim3((unsigned)segs, (unsigned)((a.h_kv + a.heads_per_cta - 1) / a.heads_per_cta));
}

}  // namespace quest
