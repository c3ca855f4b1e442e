// Cache append that norms query and key heads, rotates them and writes keys and
// values into their pages, as they are or as E4M3 codes, and folds the keys as
// stored into the page summaries.
//
// Mathematics, per head of D dims: r = rsqrt(mean(x^2) + eps), y = x r w, the
// rotation of rope_append.cu, one rounding to the cache's type. E4M3: a power
// of two per token and KV head, the least 2^e with every |y| <= 448 2^e, codes
// y 2^-e to the nearest. Powers of two lose nothing beside the rounding of the
// codes themselves (they move no mantissa), and leave every stored value an
// fp16 number, which the fp16 summary then bounds without a rounding of its own.
//
// Split. As rope_append.cu: a CTA takes the new tokens of one (request, page)
// and a run of KV heads with their query heads, a warp one head at a time, a
// lane two 16-byte pieces of every TG-th token, so that a head's sum of squares
// and largest magnitude are joined by a few shuffles. E4M3 values: a warp takes
// 16 tokens of a head at once, a lane four tokens of 4 D / 32 dims, which are
// the 16-byte chunks of the record; where the page is not complete each token's
// bytes are stored by themselves (a code's byte belongs to one token).
//
// Bound: HBM for prompts, if the warps' arithmetic keeps out of the way: with 16
// warps per SM (registers) a row's chain norm - rotate - quantise
// is as long as its copy. So the next step's rows are fetched while one is
// treated, the tokens of a step are treated side by side, pairs in packed fp32,
// boxes as fp16 minima and maxima, not as ordered keys. Decode steps: latency.
//
// Measured: 65536 tokens, 8 KV heads of 4, normed, fp16 with E4M3 summaries 248
// us, 6500 GB/s (96% of the copy rate; 357 with loads, chain and stores in turn,
// 325 with the next step fetched, 278 with a step's tokens side by side, 267 with
// fp16 boxes); 131072 tokens of 32 heads into E4M3, pages of 32, 826 us, 6590 GB/s
// (97%; 1196 with spills, which max.NaN on magnitudes ended). Three steps held
// instead of two: 283 instead of 267, 896 instead of 835. One token of 16 requests, 8 KV heads of 4: 3.5 us, into
// E4M3 4.1. 2048 tokens, one wave of CTAs: 14.5 us (52%), into E4M3 15.1 (46%); 64 dims,
// 3300 tokens of 32 heads of 8: 58.7 (68%), whose steps have half the bytes.
#pragma once

#include "append_parts.cuh"
#include "e4m3_page.cuh"
#include "quant.h"
#include "tc.cuh"
#include "tmap.h"

namespace quest {

// 16 or 8 bytes into shared memory, on the way while the warp computes.
__device__ __forceinline__ void fetch16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void fetch8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 fetched16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 fetched8(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}

// Physical page of logical page lp of request r, or -1 (reported) where the
// table or the pool has none. For the whole CTA. (rope_append.cu has the same lines
// in place: sharing them made that kernel slower.)
__device__ __forceinline__ int page_of(const RopeAppendArgs& a, int r, int lp) {
  const int entry = a.page_indptr[r] + lp;
  if (lp >= a.page_indptr[r + 1] - a.page_indptr[r] || entry >= a.nnz) {
    if (threadIdx.x == 0) report(a.err, QUEST_DEVERR_TABLE_RANGE);
    return -1;
  }
  const int pp = a.page_indices[entry];
  if (pp < 0 || pp >= a.n_phys) {
    if (threadIdx.x == 0) report(a.err, QUEST_DEVERR_PAGE_RANGE);
    return -1;
  }
  return pp;
}

// Neighbours (2e, 2e + 1) of the two pieces in a row.
template <typename T>
__device__ __forceinline__ void turn_neighbours(float* x, const float* cs, const float* sn) {
  constexpr int VEC = Elem<T>::kVec;
#pragma unroll
  for (int e = 0; e < VEC; e += 4) {
    const float4 c4 = *reinterpret_cast<const float4*>(cs + e), s4 = *reinterpret_cast<const float4*>(sn + e);
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const float a = x[2 * (e + h)], b = x[2 * (e + h) + 1];
      x[2 * (e + h)] = a * c[h] - b * s[h];
      x[2 * (e + h) + 1] = b * c[h] + a * s[h];
    }
  }
}

// The rotation of a lane's two pieces v. Pairs of the halves are turned two at a
// time (packed arithmetic; sn is negated for it), neighbours one by one.
template <typename T, bool IL>
__device__ __forceinline__ void turn_pieces(float* v, const float* cs, const float* sn) {
  constexpr int VEC = Elem<T>::kVec;
  if constexpr (IL) {
    turn_neighbours<T>(v, cs, sn);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      const float4 c4 = *reinterpret_cast<const float4*>(cs + e), s4 = *reinterpret_cast<const float4*>(sn + e);
#pragma unroll
      for (int h = 0; h < 4; h += 2) {
        const float2 c = h ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y);
        const float2 s = h ? make_float2(s4.z, s4.w) : make_float2(s4.x, s4.y);
        float* pa = v + e + h;
        float* pb = v + VEC + e + h;
        const float2 x = make_float2(pa[0], pa[1]), y = make_float2(pb[0], pb[1]);
        const float2 p = fma2(x, c, mul2(y, s)), q = fma2(mul2(x, s), both(-1.f), mul2(y, c));
        pa[0] = p.x; pa[1] = p.y;
        pb[0] = q.x; pb[1] = q.y;
      }
    }
  }
}

// Sixteen tokens' values of one head, fetched by fetch8 (token k, dims 32 i +
// ..: place k (D / 32) + i), as codes into the record's V chunks. Returns
// whether one could not be kept as it is.
template <int D>
__device__ __forceinline__ bool store_values(uint32_t src, uint8_t* rec, int S, int sub, int slot0, int ntok,
                                             int lane) {
  const int g = lane >> 2, t = lane & 3;
  uint2 x[4][D / 32];
  bool there[4], over = false;
  uint32_t top2[2];                             // of tokens 0, 1 and of 2, 3
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int tok = sub * 16 + (k >> 1) * 8 + 2 * t + (k & 1) - slot0;
    there[k] = tok >= 0 && tok < ntok;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      x[k][i] = make_uint2(0u, 0u);
      if (there[k]) x[k][i] = fetched8(src + (k * (D / 32) + i) * 256);
    }
  }
  auto largest = [&] {
    uint32_t m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      m[k] = 0u;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) m[k] = max_magnitude(max_magnitude(m[k], x[k][i].x), x[k][i].y);
      m[k] = max(m[k] & 0xffffu, m[k] >> 16);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      top2[k] = m[2 * k] | m[2 * k + 1] << 16;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) top2[k] = __vmaxu2(top2[k], __shfl_xor_sync(FULL, top2[k], o));
    }
  };
  largest();
  if (__any_sync(FULL, __vcmpgtu2(__vmaxu2(top2[0], top2[1]), kScaleTop * 0x00010001u) != 0u)) {
    over = true;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) x[k][i] = make_uint2(keepable(x[k][i].x), keepable(x[k][i].y));
    largest();
  }
  int ex[4];
  uint32_t down[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    ex[k] = scale_exponent(top2[k >> 1] >> 16 * (k & 1) & 0xffffu);
    down[k] = pow2_h2(-ex[k]);
  }
  const bool all = there[0] && there[1] && there[2] && there[3];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    uint32_t c[4];                              // a token's codes of four dims
#pragma unroll
    for (int k = 0; k < 4; ++k)
      c[k] = e4m3_codes(mul_h2(x[k][i].x, down[k])) | e4m3_codes(mul_h2(x[k][i].y, down[k])) << 16;
    uint8_t* at = rec + S * D + ((sub * (D / 32) + i) * 32 + lane) * 16;
    if (all) {                                  // a dim's codes of four tokens
      const uint32_t l01 = __byte_perm(c[0], c[1], 0x5140), h01 = __byte_perm(c[0], c[1], 0x7362);
      const uint32_t l23 = __byte_perm(c[2], c[3], 0x5140), h23 = __byte_perm(c[2], c[3], 0x7362);
      st_v4(at, make_uint4(__byte_perm(l01, l23, 0x5410), __byte_perm(l01, l23, 0x7632),
                           __byte_perm(h01, h23, 0x5410), __byte_perm(h01, h23, 0x7632)));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (there[k])
#pragma unroll
          for (int e = 0; e < 4; ++e) at[4 * e + k] = (uint8_t)(c[k] >> 8 * e);
    }
  }
  if (g == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (there[k]) rec[2 * S * D + S + sub * 16 + (k >> 1) * 8 + 2 * t + (k & 1)] = (uint8_t)(127 + ex[k]);
  }
  return over;
}

// A page's box over a lane's two pieces, as it is kept in registers: for fp16
// the numbers themselves (min.f16x2 and max.f16x2 order -0 below +0, as the
// summaries do), for fp32 the keys of Box.
template <typename T> struct Bounds {
  Box<T, false> a, b;
  __device__ __forceinline__ void clear() { a.clear(); b.clear(); }
  __device__ __forceinline__ void fold(uint4 x, uint4 y) { a.fold(x); b.fold(y); }
  __device__ __forceinline__ void join(int o) { a.join(o); b.join(o); }
  __device__ __forceinline__ void load(const char* lo, const char* hi, int ca, int cb) {
    a.load(lo + ca * sizeof(T), hi + ca * sizeof(T));
    b.load(lo + cb * sizeof(T), hi + cb * sizeof(T));
  }
  __device__ __forceinline__ void store(char* lo, char* hi, int ca, int cb) const {
    bool none = false;
    a.store(lo + ca * sizeof(T), hi + ca * sizeof(T), none);
    b.store(lo + cb * sizeof(T), hi + cb * sizeof(T), none);
  }
};
template <> struct Bounds<__half> {
  uint32_t mn[8], mx[8];
  __device__ __forceinline__ static uint32_t least(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ __forceinline__ static uint32_t most(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < 8; ++e) { mn[e] = 0x7c007c00u; mx[e] = 0xfc00fc00u; }
  }
  __device__ __forceinline__ void fold(uint4 x, uint4 y) {
    const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) { mn[e] = least(mn[e], v[e]); mx[e] = most(mx[e], v[e]); }
  }
  __device__ __forceinline__ void join(int o) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mn[e] = least(mn[e], __shfl_xor_sync(FULL, mn[e], o));
      mx[e] = most(mx[e], __shfl_xor_sync(FULL, mx[e], o));
    }
  }
  __device__ __forceinline__ void put(uint32_t* to, uint4 v) { to[0] = v.x; to[1] = v.y; to[2] = v.z; to[3] = v.w; }
  __device__ __forceinline__ void load(const char* lo, const char* hi, int ca, int cb) {
    put(mn, ld_v4(lo + ca * 2));
    put(mn + 4, ld_v4(lo + cb * 2));
    put(mx, ld_v4(hi + ca * 2));
    put(mx + 4, ld_v4(hi + cb * 2));
  }
  __device__ __forceinline__ void store(char* lo, char* hi, int ca, int cb) const {
    st_v4(lo + ca * 2, make_uint4(mn[0], mn[1], mn[2], mn[3]));
    st_v4(lo + cb * 2, make_uint4(mn[4], mn[5], mn[6], mn[7]));
    st_v4(hi + ca * 2, make_uint4(mx[0], mx[1], mx[2], mx[3]));
    st_v4(hi + cb * 2, make_uint4(mx[4], mx[5], mx[6], mx[7]));
  }
  // E4M3 summaries: codes to fp16 is exact, and outward again on the way back.
  __device__ __forceinline__ void load_codes(const char* lo, const char* hi, int ca, int cb) {
    auto four = [&](uint32_t* to, const char* at) {
      put(to, Box<__half, true>::decode(*reinterpret_cast<const uint2*>(at)));
    };
    four(mn, lo + ca);
    four(mn + 4, lo + cb);
    four(mx, hi + ca);
    four(mx + 4, hi + cb);
  }
  // The token groups share the conversions: min and max of the two pieces.
  __device__ __forceinline__ void store_codes(char* lo, char* hi, int ca, int cb, int tg, bool& ovf) const {
    const bool up = tg & 1, second = tg & 2;
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = up ? (second ? mx[4 + e] : mx[e]) : (second ? mn[4 + e] : mn[e]);
      if (up) v[e] ^= 0x80008000u;              // upwards is downwards of the negative
    }
    uint2 c = make_uint2(e4m3_floor4(v[0], v[1], ovf), e4m3_floor4(v[2], v[3], ovf));
    if (up) {
      c.x ^= __vcmpne4(c.x, 0u) & 0x80808080u;  // a zero stays +0
      c.y ^= __vcmpne4(c.y, 0u) & 0x80808080u;
    }
    if (tg < 4) st_v2((up ? hi : lo) + (second ? cb : ca), c);
  }
};

// A row of a CTA's work is the tokens of one head, a step of it 16 tokens (fp32,
// 128 dims: 8), or with FEW (calls of a few tokens per request) no more than
// stand side by side. A warp's next step is always on its way to shared memory
// while it treats the one before. A lane reads back what it fetched itself, so
// nothing but its own copies is waited for.
template <typename T, int D, bool E4, bool FEW> struct AppendStep {
  static constexpr int PC = D * sizeof(T) / 32; // lanes per token: pairs of 16-byte pieces
  static constexpr int TG = 32 / PC;            // tokens side by side
  static constexpr int U = FEW ? 1 : TG < 8 ? 4 : 2;   // and one after the other
  static constexpr uint32_t BYTES = E4 ? 16 * D * 2 : U * 1024;   // (E4M3 values: always 16 tokens)
  static constexpr int HELD = BYTES < 4096 ? 3 : 2;    // steps in shared memory per warp
};

template <typename T, int D, bool E4, bool F8, bool IL, bool FEW, int NT>
__global__ void __launch_bounds__(NT, 512 / NT) norm_append_kernel(const NormAppendArgs p) {
  static_assert(sizeof(T) == 2 || !(E4 || F8), "8-bit codes are made of fp16 rows");
  constexpr int VEC = Elem<T>::kVec;
  using Step = AppendStep<T, D, E4, FEW>;
  constexpr int PC = Step::PC, TG = Step::TG, U = Step::U, NW = NT / 32;
  extern __shared__ __align__(16) uint8_t s_fetch[];
  __shared__ __align__(16) float s_cos[kMaxPage * D / 2], s_sin[kMaxPage * D / 2];
  const RopeAppendArgs& a = p.a;

  int r, j;
  if (!touched_page<NT>(a, blockIdx.x, &r, &j)) return;
  const int S = a.page_size, first = a.append_indptr[r], pos0 = a.seq_lens_before[r];
  const int n_r = a.append_indptr[r + 1] - first;
  const int lp = pos0 / S + j;
  const int t_begin = max(pos0, lp * S), t_end = min(pos0 + n_r, (lp + 1) * S);
  const int row0 = first + (t_begin - pos0);
  const int ntok = min(t_end - t_begin, a.n_new - row0);
  if (ntok <= 0) return;
  const int half = a.rotary_dim / 2;
  const int slot0 = t_begin - lp * S;

  const int h0 = blockIdx.y * a.heads_per_cta, h1 = min(a.h_kv, h0 + a.heads_per_cta);
  const int nh = h1 - h0;
  const int qn = a.q ? nh * a.group : 0;        // rows: queries, then keys, then values
  const int v_rows = E4 ? S / 16 : 1;           // E4M3 values: 16 tokens at a time
  const int rows = qn + (1 + v_rows) * nh;

  const int lane = threadIdx.x & 31, it = threadIdx.x % PC, tg = lane / PC;
  int ca = 2 * it, cb = 2 * it + 1;             // the lane's pieces, and whether they turn
  bool turn = ca * VEC < a.rotary_dim;
  if (!IL) {
    turn = it * VEC < half;
    if (turn) { ca = it; cb = it + half / VEC; }
  }
  ca *= VEC;
  cb *= VEC;
  const uint32_t ring = smem_u32(s_fetch) + (threadIdx.x / 32) * Step::HELD * Step::BYTES + lane * 16;

  // Start the copies of a row's tokens from t0 on into place `buf`.
  auto fetch = [&](int row, int t0, int buf) {
    const uint32_t dst = ring + buf * Step::BYTES;
    if (row >= rows) {                          // the warp's last step has none behind it
    } else if (E4 && row >= qn + nh) {
      const int i0 = row - qn - nh, h = h0 + i0 / v_rows, sub = i0 % v_rows;
      const T* src = static_cast<const T*>(a.v_new) + row0 * a.v_stride + h * D + 4 * (lane >> 2);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int tok = sub * 16 + (k >> 1) * 8 + 2 * (lane & 3) + (k & 1) - slot0;
        if (tok >= 0 && tok < ntok)
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            fetch8(dst - lane * 8 + (k * (D / 32) + i) * 256, src + tok * a.v_stride + 32 * i);
      }
    } else {
      const T* src;
      int64_t stride;
      if (row < qn) {
        stride = a.q_stride;
        src = static_cast<const T*>(a.q) + (h0 * a.group + row) * D;
      } else if (row < qn + nh) {
        stride = a.k_stride;
        src = static_cast<const T*>(a.k_new) + (h0 + row - qn) * D;
      } else {
        stride = a.v_stride;
        src = static_cast<const T*>(a.v_new) + (h0 + row - qn - nh) * D;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * TG + tg;
        if (t < ntok) {
          fetch16(dst + u * 1024, src + (row0 + t) * stride + ca);
          fetch16(dst + u * 1024 + 512, src + (row0 + t) * stride + cb);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // The step behind (row, t0).
  auto behind = [&](int& row, int& t0) {
    if ((E4 && row >= qn + nh) || t0 + U * TG >= ntok) {
      row += NW;
      t0 = 0;
    } else {
      t0 += U * TG;
    }
  };
  int next_row = threadIdx.x / 32, next_t0 = 0;
#pragma unroll
  for (int k = 0; k < Step::HELD - 1; ++k) {
    fetch(next_row, next_t0, k);
    behind(next_row, next_t0);
  }

  if (half > 0) {
    const int jj = threadIdx.x % half;
    const unsigned long long f = turn_fraction(a.inv_freq[jj]);
    for (int t = threadIdx.x / half; t < ntok && threadIdx.x < NT / half * half; t += NT / half) {
      const int pos = a.positions ? a.positions[row0 + t] : t_begin + t;
      const int angle = (int)(((unsigned long long)(long long)pos * f) >> 32);   // half turns in 2^-31
      float sn, cs;
      sincospif((float)angle * 0x1p-31f, &sn, &cs);
      s_cos[t * (D / 2) + jj] = cs;
      s_sin[t * (D / 2) + jj] = IL ? sn : -sn;
    }
  }
  const int pp = page_of(a, r, lp);             // without a page the queries are treated all the same
  __syncthreads();

  const bool fresh = slot0 == 0;
  const size_t page = (size_t)max(pp, 0) * a.h_kv;
  const size_t rec = record_bytes(S, D);
  constexpr size_t SE = F8 ? 1 : sizeof(T);     // bytes of a summary element
  bool ovf = false;
  Bounds<T> box;                                // of the row of keys in hand

  // The U TG tokens of a step (zeros where there is none), normed (with a
  // weight) and turned, as they are stored. All of them at once: what one
  // token's chain of sums and shuffles waits for, the others fill.
  auto treat = [&](uint32_t src, int t0, const float* weight, uint4 (&x)[U], uint4 (&y)[U]) {
    float f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u] = y[u] = make_uint4(0u, 0u, 0u, 0u);
      f[u] = 1.f;
      if (t0 + u * TG + tg < ntok) {
        x[u] = fetched16(src + u * 1024);
        y[u] = fetched16(src + u * 1024 + 512);
      }
    }
    float w[2 * VEC];
    if (weight) {                               // of the whole warp
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        *reinterpret_cast<float4*>(w + e) = *reinterpret_cast<const float4*>(weight + ca + e);
        *reinterpret_cast<float4*>(w + VEC + e) = *reinterpret_cast<const float4*>(weight + cb + e);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[2 * VEC];
        unpack16<T>(x[u], v);
        unpack16<T>(y[u], v + VEC);
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 2 * VEC; e += 2) ss = fma2(make_float2(v[e], v[e + 1]), make_float2(v[e], v[e + 1]), ss);
        f[u] = ss.x + ss.y;
      }
#pragma unroll
      for (int o = 1; o < PC; o <<= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) f[u] += __shfl_xor_sync(FULL, f[u], o);
#pragma unroll
      for (int u = 0; u < U; ++u) f[u] = rsqrtf(fmaf(f[u], 1.f / D, p.eps));
    }
    if (weight || turn) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[2 * VEC];
        unpack16<T>(x[u], v);
        unpack16<T>(y[u], v + VEC);
        if (weight) {
#pragma unroll
          for (int e = 0; e < 2 * VEC; e += 2) {
            const float2 n = mul2(make_float2(v[e], v[e + 1]), mul2(make_float2(w[e], w[e + 1]), both(f[u])));
            v[e] = n.x;
            v[e + 1] = n.y;
          }
        }
        if (turn) {
          const int at = min(t0 + u * TG + tg, ntok - 1) * (D / 2) + it * VEC;
          turn_pieces<T, IL>(v, s_cos + at, s_sin + at);
        }
        x[u] = Pack<T>::pack(v);
        y[u] = Pack<T>::pack(v + VEC);
      }
    }
    __syncwarp();
  };

  int buf = 0;
  for (int row = threadIdx.x / 32, t0 = 0; row < rows; behind(row, t0)) {
    fetch(next_row, next_t0, buf == 0 ? Step::HELD - 1 : buf - 1);
    behind(next_row, next_t0);
    asm volatile("cp.async.wait_group %0;" :: "n"(Step::HELD - 1) : "memory");
    const uint32_t src = ring + buf * Step::BYTES;
    if (++buf == Step::HELD) buf = 0;
    if (row < qn + nh) {
      if (row >= qn && pp < 0) break;
      const int h = row < qn ? h0 * a.group + row : h0 + row - qn;
      const float* weight = row < qn ? p.q_weight : p.k_weight;
      if (weight && (row < qn ? p.q_per_head : p.k_per_head)) weight += h * D;
      uint4 x[U], y[U];
      treat(src, t0, weight, x, y);
      if (row < qn) {
        const int64_t out_stride = (int64_t)a.h_kv * a.group * D;
        T* out = static_cast<T*>(a.q_out) + (row0 + t0 + tg) * out_stride + h * D;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (t0 + u * TG + tg < ntok) {
            st_v4(out + u * TG * out_stride + ca, x[u]);
            st_v4(out + u * TG * out_stride + cb, y[u]);
          }
      } else {
        char* sm = static_cast<char*>(a.summary) + (page + h) * 2 * D * SE;
        if (t0 == 0) {
          if (fresh || tg != 0) box.clear();
          else if constexpr (F8) box.load_codes(sm, sm + D, ca, cb);
          else box.load(sm, sm + D * SE, ca, cb);
        }
        if constexpr (E4) {
          uint8_t* to = static_cast<uint8_t*>(a.k_pool) + (page + h) * rec;
          uint32_t top[U];
          auto largest = [&] {
#pragma unroll
            for (int u = 0; u < U; ++u) {
              uint32_t m = max_magnitude(max_magnitude(0u, x[u].x), x[u].y);
              m = max_magnitude(max_magnitude(m, x[u].z), x[u].w);
              m = max_magnitude(max_magnitude(m, y[u].x), y[u].y);
              m = max_magnitude(max_magnitude(m, y[u].z), y[u].w);
              top[u] = max(m & 0xffffu, m >> 16);
            }
#pragma unroll
            for (int o = 1; o < PC; o <<= 1)
#pragma unroll
              for (int u = 0; u < U; ++u) top[u] = max(top[u], __shfl_xor_sync(FULL, top[u], o));
          };
          largest();
          uint32_t most = 0u;
#pragma unroll
          for (int u = 0; u < U; ++u) most = max(most, top[u]);
          if (__any_sync(FULL, most > kScaleTop)) {
            ovf = true;
#pragma unroll
            for (int u = 0; u < U; ++u) {
              x[u] = make_uint4(keepable(x[u].x), keepable(x[u].y), keepable(x[u].z), keepable(x[u].w));
              y[u] = make_uint4(keepable(y[u].x), keepable(y[u].y), keepable(y[u].z), keepable(y[u].w));
            }
            largest();
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int ex = scale_exponent(top[u]), t = t0 + u * TG + tg;
            const uint32_t down = pow2_h2(-ex), up = pow2_h2(ex);
            const uint32_t v[8] = {x[u].x, x[u].y, x[u].z, x[u].w, y[u].x, y[u].y, y[u].z, y[u].w};
            uint32_t c[4], kept[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t lo = e4m3_codes(mul_h2(v[2 * e], down)), hi = e4m3_codes(mul_h2(v[2 * e + 1], down));
              c[e] = lo | hi << 16;
              kept[2 * e] = mul_h2(e4m3_pair(lo), up);
              kept[2 * e + 1] = mul_h2(e4m3_pair(hi), up);
            }
            if (t < ntok) {
              const int slot = slot0 + t;
              st_v2(to + k_code_at(S, slot, ca), make_uint2(c[0], c[1]));
              st_v2(to + k_code_at(S, slot, cb), make_uint2(c[2], c[3]));
              if (it == 0) to[2 * S * D + slot] = (uint8_t)(127 + ex);
              box.fold(make_uint4(kept[0], kept[1], kept[2], kept[3]), make_uint4(kept[4], kept[5], kept[6], kept[7]));
            }
          }
        } else {
          T* to = static_cast<T*>(a.k_pool) + ((page + h) * S + slot0 + t0 + tg) * D;
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (t0 + u * TG + tg < ntok) {
              st_v4(to + u * TG * D + ca, x[u]);
              st_v4(to + u * TG * D + cb, y[u]);
              box.fold(x[u], y[u]);
            }
        }
        if (t0 + U * TG >= ntok) {
          __syncwarp();
#pragma unroll
          for (int o = PC; o < 32; o <<= 1) box.join(o);
          if constexpr (F8) box.store_codes(sm, sm + D, ca, cb, tg, ovf);
          else if (tg == 0) box.store(sm, sm + D * SE, ca, cb);
        }
      }
    } else if (pp < 0) {
      break;
    } else if constexpr (E4) {
      const int i0 = row - qn - nh, h = h0 + i0 / v_rows, sub = i0 % v_rows;
      if (slot0 + ntok > sub * 16 && slot0 < sub * 16 + 16)
        ovf |= store_values<D>(src - lane * 8, static_cast<uint8_t*>(a.k_pool) + (page + h) * rec, S, sub,
                               slot0, ntok, lane);
    } else {
      T* to = static_cast<T*>(a.v_pool) + ((page + h0 + row - qn - nh) * S + slot0) * D;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * TG + tg;
        if (t < ntok) {
          st_v4(to + t * D + ca, fetched16(src + u * 1024));
          st_v4(to + t * D + cb, fetched16(src + u * 1024 + 512));
        }
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if ((E4 || F8) && ovf) report(a.err, QUEST_DEVERR_FP8_RANGE);
}

template <typename T, int D, bool E4, bool F8, bool FEW, int NT>
cudaError_t launch_norm_append_n(const NormAppendArgs& p, dim3 grid, cudaStream_t s) {
  using Step = AppendStep<T, D, E4, FEW>;
  constexpr int smem = NT / 32 * Step::HELD * Step::BYTES;
  auto kernel = p.a.interleaved ? norm_append_kernel<T, D, E4, F8, true, FEW, NT>
                                : norm_append_kernel<T, D, E4, F8, false, FEW, NT>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, NT, smem, s>>>(p);
  return cudaGetLastError();
}
// Up to four new tokens per request, on average: a step goes through no more of
// them than stand side by side (a token of 16 requests 4.3 -> 3.5 us, of 200
// requests 15 -> 9; a branch inside one kernel made it too large: 65536 tokens
// 248 -> 260). Where one request brings a chunk this may be the slower way (250
// requests of one token and one of 700: 18.8 us, 17.6 with full steps; 1000 and one
// of 3000: 52 and 62): the host knows the average alone.
// Many CTAs: four warps each, four of them per SM, whose starts the others hide
// (65536 tokens, 8 KV heads of 4: 267 us with eight warps, 248 with four). Where the
// device is not full eight warps get through a page sooner.
template <typename T, int D, bool E4, bool F8>
cudaError_t launch_norm_append_t(const NormAppendArgs& p, dim3 grid, int sms, cudaStream_t s) {
  const bool many = (long long)grid.x * grid.y > 4LL * sms;
  if (p.a.n_new <= 4LL * p.a.batch)
    return many ? launch_norm_append_n<T, D, E4, F8, true, 128>(p, grid, s)
                : launch_norm_append_n<T, D, E4, F8, true, 256>(p, grid, s);
  return many ? launch_norm_append_n<T, D, E4, F8, false, 128>(p, grid, s)
              : launch_norm_append_n<T, D, E4, F8, false, 256>(p, grid, s);
}

}  // namespace quest
