// Cache append with the position rotation applied on the way: rotate k, write
// k and v into their pages, fold the rotated keys into the page summaries
// (Quest page §1.2 eq (8), §3 eq (14)), rotate the queries of the same tokens.
//
// Mathematics. Pair j of a head at position p turns by p * inv_freq[j]. Only
// the fraction of a turn matters, so f = inv_freq / (2 pi) is taken once as a
// 64-bit fixed-point fraction of a turn; p * f mod 2^64 is an exact integer
// product, and its high word is the angle to 2^-32 turns, however far p is.
// cos and sin come from sincospif.
//
// Split. A page's summary has one writer: a CTA takes the new tokens of one
// (request, page) and a run of KV heads with their query heads. It fills a
// table of cos and sin for its tokens in shared memory once, then a warp takes
// one head at a time: a lane holds two 16-byte pieces (the two halves of VEC
// pairs, or two neighbouring pieces) of every TG-th token, with the min and max
// of a key's dims in registers, joined over the token groups by shuffles. HBM
// bound for prompts: every row is read and written once; decode steps are
// latency bound and spread over the KV heads.
//
// Measured (fp16, d 128): 131072 tokens of 32 heads, pages of 32, 1012 us, 6430
// GB/s (95% of the copy rate; 1220 us before the token groups, one thread then
// taking a piece through all tokens); one token of 16 requests, 8 KV heads of
// 4, E4M3 summaries, 6.2 us. Two CTAs per SM with four tokens in flight beat
// three with two (1030 and 1106 us).
#include "common.cuh"
#include "dense.h"
#include "tmap.h"

namespace quest {
namespace {

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
__device__ __forceinline__ void walk(const T* src, int64_t src_stride, T* dst, int64_t dst_stride,
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

template <typename T, int D, bool F8, bool IL, int NT>
__global__ void __launch_bounds__(NT, 512 / NT) rope_append_kernel(const RopeAppendArgs a) {
  static_assert(!F8 || sizeof(T) == 2, "E4M3 summaries take fp16 keys");
  constexpr int VEC = Elem<T>::kVec;
  constexpr int PC = D / VEC / 2;               // pairs of 16-byte pieces per head
  __shared__ __align__(16) float s_cos[kMaxPage * D / 2], s_sin[kMaxPage * D / 2];

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

  // a thread keeps its pair through the tokens
  const int jj = threadIdx.x % half;
  const unsigned long long f = turn_fraction(a.inv_freq[jj]);
  for (int t = threadIdx.x / half; t < ntok && threadIdx.x < NT / half * half; t += NT / half) {
    const int p = a.positions ? a.positions[row0 + t] : t_begin + t;
    const int turn = (int)(((unsigned long long)(long long)p * f) >> 32);   // half turns in 2^-31
    float sn, cs;
    sincospif((float)turn * 0x1p-31f, &sn, &cs);
    s_cos[t * (D / 2) + jj] = cs;
    s_sin[t * (D / 2) + jj] = sn;
  }

  // the page; without one the queries are rotated all the same
  const int entry = a.page_indptr[r] + lp;
  int pp = -1;
  if (lp >= a.page_indptr[r + 1] - a.page_indptr[r] || entry >= a.nnz) {
    if (threadIdx.x == 0) report(a.err, QUEST_DEVERR_TABLE_RANGE);
  } else {
    pp = a.page_indices[entry];
    if (pp < 0 || pp >= a.n_phys) {
      if (threadIdx.x == 0) report(a.err, QUEST_DEVERR_PAGE_RANGE);
      pp = -1;
    }
  }
  __syncthreads();

  const int h0 = blockIdx.y * a.heads_per_cta, h1 = min(a.h_kv, h0 + a.heads_per_cta);
  const int nh = h1 - h0;
  const int qn = a.q ? nh * a.group : 0;        // rows: queries, then keys, then values
  const int slot0 = t_begin - lp * S;
  const bool fresh = slot0 == 0;
  const size_t page = (size_t)max(pp, 0) * a.h_kv;
  constexpr size_t SE = F8 ? 1 : sizeof(T);     // bytes of a summary element
  bool ovf = false;

  // a warp takes a row at a time: its pieces, at TG tokens side by side
  constexpr int TG = 32 / PC;
  const int it = threadIdx.x % PC, tg = threadIdx.x % 32 / PC;
  // the lane's two pieces, and whether they are rotated
  int ca = 2 * it, cb = 2 * it + 1;
  bool turn = ca * VEC < a.rotary_dim;
  if (!IL) {
    turn = it * VEC < half;
    if (turn) { ca = it; cb = it + half / VEC; }
    // the others, from the rotary part on, in neighbours: 2 * it as above
  }
  ca *= VEC;
  cb *= VEC;
  const float* cs = s_cos + it * VEC;
  const float* sn = s_sin + it * VEC;
  auto turned = [&](uint4& x, uint4& y, int tok) {
    if (turn) rotate<T, IL>(x, y, cs + tok * (D / 2), sn + tok * (D / 2));
  };
  for (int row = threadIdx.x / 32; row < qn + 2 * nh; row += NT / 32) {
    if (row < qn) {
      const int h = h0 * a.group + row;
      const int64_t out_stride = (int64_t)a.h_kv * a.group * D;
      walk<T, TG>(static_cast<const T*>(a.q) + row0 * a.q_stride + h * D, a.q_stride,
                  static_cast<T*>(a.q_out) + row0 * out_stride + h * D, out_stride, ca, cb, tg, ntok,
                  turned);
    } else if (pp < 0) {
      break;
    } else if (row < qn + nh) {
      const int h = h0 + row - qn;
      char* sm = static_cast<char*>(a.summary) + (page + h) * 2 * D * SE;
      Box<T, F8> ba, bb;
      if (fresh || tg != 0) {
        ba.clear();
        bb.clear();
      } else {
        ba.load(sm + ca * SE, sm + (D + ca) * SE);
        bb.load(sm + cb * SE, sm + (D + cb) * SE);
      }
      walk<T, TG>(static_cast<const T*>(a.k_new) + row0 * a.k_stride + h * D, a.k_stride,
                  static_cast<T*>(a.k_pool) + ((page + h) * S + slot0) * D, D, ca, cb, tg, ntok,
                  [&](uint4& x, uint4& y, int tok) {
                    turned(x, y, tok);
                    ba.fold(x);
                    bb.fold(y);
                  });
      __syncwarp();
#pragma unroll
      for (int o = PC; o < 32; o <<= 1) {
        ba.join(o);
        bb.join(o);
      }
      if (tg == 0) {
        ba.store(sm + ca * SE, sm + (D + ca) * SE, ovf);
        bb.store(sm + cb * SE, sm + (D + cb) * SE, ovf);
      }
    } else {
      const int h = h0 + row - qn - nh;
      walk<T, TG>(static_cast<const T*>(a.v_new) + row0 * a.v_stride + h * D, a.v_stride,
                  static_cast<T*>(a.v_pool) + ((page + h) * S + slot0) * D, D, ca, cb, tg, ntok,
                  [](uint4&, uint4&, int) {});
    }
  }
  if (F8 && ovf) report(a.err, QUEST_DEVERR_FP8_RANGE);
}

template <typename T, int D, bool F8, int NT>
cudaError_t launch_n(const RopeAppendArgs& a, dim3 grid, cudaStream_t s) {
  if (a.interleaved) rope_append_kernel<T, D, F8, true, NT><<<grid, NT, 0, s>>>(a);
  else rope_append_kernel<T, D, F8, false, NT><<<grid, NT, 0, s>>>(a);
  return cudaGetLastError();
}

// Many CTAs of few rows: four warps each, so that more of them start at once
// (53823 tokens, one KV head of 8, E4M3: 103 us with eight warps, 76 with four;
// 65536 tokens of one head 61 and 37). From 24 rows on the two are alike, and
// where the device is not full eight warps get through a page sooner.
template <typename T, int D, bool F8>
cudaError_t launch(const RopeAppendArgs& a, dim3 grid, int sms, cudaStream_t s) {
  const int rows = a.heads_per_cta * ((a.q ? a.group : 0) + 2);
  const bool small = rows <= 16 && (long long)grid.x * grid.y > 4LL * sms;
  return small ? launch_n<T, D, F8, 128>(a, grid, s) : launch_n<T, D, F8, 256>(a, grid, s);
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs& args, cudaStream_t s) {
  RopeAppendArgs a = args;
  const int sms = sm_count();
  // a request with n new tokens touches at most ceil(n / S) + 1 pages, each
  // with one token at least
  long long segs = (long long)(a.n_new + a.page_size - 1) / a.page_size + 2LL * a.batch;
  if (segs > a.n_new) segs = a.n_new;
  // Few pages: the KV heads of one are spread over CTAs until every SM has one;
  // more CTAs only start more often (200 one-token requests of 8 KV heads: 9.5
  // us with 152 CTAs wanted, 13.6 with 608; 2048 tokens 11.5 and 19.3).
  a.heads_per_cta = a.h_kv;
  while (a.heads_per_cta > 1 && segs * ((a.h_kv + a.heads_per_cta - 1) / a.heads_per_cta) < sms)
    a.heads_per_cta = (a.heads_per_cta + 1) / 2;
  const dim3 grid((unsigned)segs, (unsigned)((a.h_kv + a.heads_per_cta - 1) / a.heads_per_cta));
  if (a.dtype == QUEST_F16 && a.summary_fp8)
    return a.head_dim == 128 ? launch<__half, 128, true>(a, grid, sms, s) : launch<__half, 64, true>(a, grid, sms, s);
  if (a.dtype == QUEST_F16)
    return a.head_dim == 128 ? launch<__half, 128, false>(a, grid, sms, s) : launch<__half, 64, false>(a, grid, sms, s);
  return a.head_dim == 128 ? launch<float, 128, false>(a, grid, sms, s) : launch<float, 64, false>(a, grid, sms, s);
}

}  // namespace quest
