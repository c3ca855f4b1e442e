// Dense decode attention: one query per request over its visible keys.
//
// Mathematics. Tiles of 16 tokens (fp32: 8) of one KV head; per tile the
// logits x of the group's heads in base 2, the running maximum m (let lag by
// up to 2^8, so that rescaling is rare), weights p = 2^(x - m + 6), l += sum p,
// o += p v. Partial (o, m, l) of the parts of a (request, KV head) are joined
// by log-sum-exp.
//
// Bound: HBM, K and V of every visible page once (2 D elements a token and KV
// head), against which the arithmetic is small even on the warp MMA.
//
// Split. The tiles of all (request, KV head) units in a row are cut into equal
// runs, one per warp, whatever the lengths: every warp streams the same number
// of bytes through a ring of its own (TMA boxes of 128-byte rows, 128-byte
// swizzle, one barrier per place) and never waits for another warp. A unit
// that lies inside one run is written at once; the parts of the others go to
// the workspace, at place (warp + unit): the two only ever grow along the
// runs, so no two parts meet there. A second kernel joins them in run order.
//
// fp16 on mma.sync m16n8k16, keys and dims as the 16 rows, the group's heads
// as (up to) the 8 columns:  S^T = K Q^T,  O^T += V^T P^T.  P is passed as two
// fp16 numbers, p = p1 + p2 to 2^-22, so the output keeps fp32 accuracy.
// fp32: plain FMA, a lane per (token, quarter of the dims) for the logits, a
// lane per dims for the values.
//
// Measured (fp16, d 128): 16 requests of 8192 to 131072 tokens, 8 KV heads of 4,
// 822 us, 6820 GB/s (100% of the copy rate); 32768 tokens of 32 heads 87.5 us (90%).
// fp32: 32768 tokens of 8 KV heads of 4, d 128, 58.6 us (4580 GB/s, 67%); 8 heads
// over 9000 to 65536 tokens, d 64, 99 us (5260 GB/s, 77%); 1000 tokens of one head
// 10 us.
#pragma once

#include "attn_mma.cuh"
#include "dense.cuh"
#include "tc.cuh"

namespace quest {

struct DecodeMaps { CUtensorMap k, v; };

struct DecodeArgs {
  DenseArgs a;
  long long* starts;        // [batch + 1] tiles before each request, all KV heads
  float* part_o;            // [warps + units, G, D]
  float2* part_ml;          // [warps + units, G]
  int32_t n_warps;
  uint32_t wait_limit;
};

template <typename T, int D> struct DecodeShape {
  static constexpr int TT = sizeof(T) == 2 ? 16 : 8;         // tokens per tile
  static constexpr int COLS = 128 / sizeof(T);               // dims per box
  static constexpr int BOXES = D / COLS;
  static constexpr uint32_t BOX = TT * 128, TILE = BOXES * BOX, STAGE = 2 * TILE;
  // 192 KB of rings. fp16, 128 dims: 8, 10 and 12 warps take 840, 823 and 819 us
  // for the ragged batch below. Half-size tiles (64 dims) are bound by their
  // instructions: 16, 20 and 24 warps take 42.1, 41.7 and 50.4 us for 64 capped
  // requests of up to 8192 tokens.
  static constexpr int WARPS = sizeof(T) == 4 ? 8 : D == 64 ? 16 : 12;
  static constexpr int STAGES = 196608 / WARPS / STAGE;
  static constexpr uint32_t SMEM = 1024 + WARPS * STAGES * STAGE;
};

// Tiles per warp: equal runs, of at least four.
__device__ __forceinline__ long long run_length(long long tiles, int n_warps) {
  const long long n = (tiles + n_warps - 1) / n_warps;
  return n < 4 ? 4 : n;
}

// The tiles of request r that hold a visible key.
struct Request { int pos, lo, hi, held, e0, tile0, tiles; };
template <int TT>
__device__ __forceinline__ Request request_of(const DenseArgs& a, int r, unsigned* err) {
  Request q;
  const int len = a.seq_lens[r];
  q.e0 = a.page_indptr[r];
  q.held = held_tokens(len, a.page_indptr[r + 1] - q.e0, a.page_size, err);
  q.pos = len - 1;
  const Seen s = seen_keys(q.pos, q.held, a.window, a.doc_starts ? a.doc_starts[r] : 0,
                           a.prefix_lens ? a.prefix_lens[r] : 0);
  q.lo = s.lo;
  q.hi = s.hi;
  q.tile0 = s.lo / TT;
  q.tiles = s.hi > s.lo ? (s.hi + TT - 1) / TT - q.tile0 : 0;
  return q;
}

// Logit -> base 2, with the call's mods (converged warps only).
struct Logit {
  float scale2, cap2, inv_cap2, slope2;
  __device__ __forceinline__ float operator()(float s, int dist) const {
    const float x = s * scale2;
    return (cap2 > 0.f ? capped(x, cap2, inv_cap2) : x) - slope2 * (float)dist;
  }
};

// Running state of the group's heads, fp16 keys. Lane: heads 2 t, 2 t + 1
// (t = lane % 4), dims 16 mt + lane / 4 and + 8.
template <int D> struct WarpF16 {
  using T = __half;
  static constexpr int KT = D / 16;
  uint32_t qb[KT][2];
  float m[2], l[2], acc[KT][4], sum[KT][4];
  float slope2[2];
  int since;                // tiles in acc

  // The tensor core's accumulation truncates: a long chain would lose a bit
  // per doubling, always downwards. acc takes eight tiles, then goes to sum.
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) { sum[k][c] += acc[k][c]; acc[k][c] = 0.f; }
    since = 0;
  }

  __device__ __forceinline__ void begin(const DenseArgs& a, int r, int g, int lane, float*) {
    const int head = lane >> 2, t = lane & 3;
    const __half* q = static_cast<const __half*>(a.q) + ((size_t)r * a.h_kv * a.group + g * a.group + head) * D;
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        qb[k][i] = head < a.group ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8 * i + 2 * t) : 0u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      slope2[i] = a.slopes && 2 * t + i < a.group ? a.slopes[g * a.group + 2 * t + i] * LOG2E : 0.f;
    }
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) sum[k][c] = acc[k][c] = 0.f;
    since = 0;
  }

  // tokens tok0 .. tok0 + 15 of the tile in shared memory at k_s and v_s
  __device__ __forceinline__ void tile(const DenseArgs& a, const Request& rq, int tok0, uint32_t k_s,
                                       uint32_t v_s, const float*, float scale2, int lane) {
    const int r8 = lane & 7, mat = lane >> 3, t = lane & 3;
    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
    {
      const int row = r8 + 8 * (mat & 1);
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        const uint32_t at = k_s + (k >> 2) * 2048 + row * 128 + ((((k & 3) * 2 + (mat >> 1)) ^ r8) << 4);
        uint32_t a0, a1, a2, a3;
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3) : "r"(at));
        if (k & 1) mma_f16_16816(s1, a0, a1, a2, a3, qb[k][0], qb[k][1]);
        else mma_f16_16816(s0, a0, a1, a2, a3, qb[k][0], qb[k][1]);
      }
    }
    const int ta = tok0 + (lane >> 2), tb = ta + 8;
    float x[4];
    if (a.softcap > 0.f || a.slopes) {
      const float cap2 = a.softcap * LOG2E, inv = 1.f / cap2;
      const Logit f0{scale2, cap2, inv, slope2[0]}, f1{scale2, cap2, inv, slope2[1]};
      const int da = abs(rq.pos - ta), db = abs(rq.pos - tb);
      x[0] = f0(s0[0] + s1[0], da);
      x[1] = f1(s0[1] + s1[1], da);
      x[2] = f0(s0[2] + s1[2], db);
      x[3] = f1(s0[3] + s1[3], db);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = (s0[c] + s1[c]) * scale2;
    }
    const bool edge = tok0 < rq.lo || tok0 + 16 > rq.hi;
    if (edge) {
      if (ta < rq.lo || ta >= rq.hi) x[0] = x[1] = -INFINITY;
      if (tb < rq.lo || tb >= rq.hi) x[2] = x[3] = -INFINITY;
    }
    float mx[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
    if (__any_sync(FULL, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
      settle();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(FULL, mx[i], o));
        if (mx[i] > m[i]) {
          const float f = ex2(m[i] - mx[i]);           // first maximum: 0, and o and l are 0
          m[i] = mx[i];
          l[i] *= f;
#pragma unroll
          for (int k = 0; k < KT; ++k) { sum[k][i] *= f; sum[k][2 + i] *= f; }
        }
      }
    }
    uint32_t hi[2], lo[2];
    const float b0 = m[0] == -INFINITY ? 0.f : m[0] - 6.f, b1 = m[1] == -INFINITY ? 0.f : m[1] - 6.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float pa = ex2(x[2 * i] - b0), pb = ex2(x[2 * i + 1] - b1);
      l[0] += pa;
      l[1] += pb;
      const __half2 h = __floats2half2_rn(pa, pb);
      const float2 back = __half22float2(h);
      const __half2 rest = __floats2half2_rn(pa - back.x, pb - back.y);
      asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(hi[i]) : "r"(*reinterpret_cast<const uint32_t*>(&h)));
      asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(lo[i]) : "r"(*reinterpret_cast<const uint32_t*>(&rest)));
    }
    // values of slots without a token may be anything (0 * NaN is NaN): their
    // halves of V^T are cleared. k index of a half: 2 t, 2 t + 1 (+ 8)
    uint32_t z0 = 0xffffffffu, z1 = 0xffffffffu;
    if (tok0 + 16 > rq.held) {
      const int n = rq.held - tok0;
      z0 = (2 * t < n ? 0xffffu : 0u) | (2 * t + 1 < n ? 0xffff0000u : 0u);
      z1 = (2 * t + 8 < n ? 0xffffu : 0u) | (2 * t + 9 < n ? 0xffff0000u : 0u);
    }
    const int row = r8 + 8 * (mat >> 1);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const uint32_t at = v_s + (k >> 2) * 2048 + row * 128 + ((((k & 3) * 2 + (mat & 1)) ^ r8) << 4);
      uint32_t a0, a1, a2, a3;
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                   : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3) : "r"(at));
      a0 &= z0; a1 &= z0; a2 &= z1; a3 &= z1;
      mma_f16_16816(acc[k], a0, a1, a2, a3, hi[0], hi[1]);
      mma_f16_16816(acc[k], a0, a1, a2, a3, lo[0], lo[1]);
    }
    if (++since == 8) settle();
  }

  // The state as o (times `whole ? 1 / l : 1`), m and l of head i, dims 16 k + ..
  template <typename F>
  __device__ __forceinline__ void finish(const DenseArgs& a, bool whole, int lane, F put) {
    const int t = lane & 3;
    settle();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) l[i] += __shfl_xor_sync(FULL, l[i], o);
      const int head = 2 * t + i;
      if (head < a.group) {
        const float f = whole ? (l[i] > 0.f ? 1.f / l[i] : 0.f) : 1.f;
        float* o = put(head, m[i], l[i], (lane >> 2) == 0);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          o[16 * k + (lane >> 2)] = sum[k][i] * f;
          o[16 * k + (lane >> 2) + 8] = sum[k][2 + i] * f;
        }
      }
    }
  }
};

// The same for fp32 keys. Logits: token lane % 8, chunks lane / 8 + 4 i of
// four dims (conflict free under the swizzle), q in shared memory; values:
// D / 32 dims per lane.
template <int D, int G> struct WarpF32 {
  using T = float;
  static constexpr int E = D / 32;
  float m[G], l[G], acc[G][E];
  float slope2[G];

  __device__ __forceinline__ void begin(const DenseArgs& a, int r, int g, int lane, float* qs) {
    const float* q = static_cast<const float*>(a.q) + ((size_t)r * a.h_kv + g) * G * D;
    __syncwarp();
    for (int i = lane; i < G * D; i += 32) qs[i] = q[i];
    __syncwarp();
#pragma unroll
    for (int h = 0; h < G; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
      slope2[h] = a.slopes ? a.slopes[g * G + h] * LOG2E : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[h][e] = 0.f;
    }
  }

  __device__ __forceinline__ void tile(const DenseArgs& a, const Request& rq, int tok0, uint32_t k_s,
                                       uint32_t v_s, const float* qs, float scale2, int lane) {
    const int tok = lane & 7, part = lane >> 3;
    float s[G];
#pragma unroll
    for (int h = 0; h < G; ++h) s[h] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int c = part + 4 * i;                      // of D / 4 chunks of 16 bytes
      float k[4];
      lds4(k_s + (c >> 3) * 1024 + tok * 128 + (((c & 7) ^ tok) << 4), k);
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float4 q = *reinterpret_cast<const float4*>(qs + h * D + c * 4);
        s[h] = fmaf(q.x, k[0], fmaf(q.y, k[1], fmaf(q.z, k[2], fmaf(q.w, k[3], s[h]))));
      }
    }
    const int at = tok0 + tok, dist = abs(rq.pos - at);
    const bool see = at >= rq.lo && at < rq.hi;
    const float cap2 = a.softcap * LOG2E, inv_cap2 = 1.f / cap2;
    float p[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      s[h] += __shfl_xor_sync(FULL, s[h], 8);
      s[h] += __shfl_xor_sync(FULL, s[h], 16);
      const Logit f{scale2, cap2, inv_cap2, slope2[h]};
      const float y = f(s[h], dist), x = see ? y : -INFINITY;
      if (__any_sync(FULL, x > m[h] + 8.f)) {
        float mx = x;
#pragma unroll
        for (int o = 1; o <= 4; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
        if (mx > m[h]) {
          const float w = ex2(m[h] - mx);
          m[h] = mx;
          l[h] *= w;
#pragma unroll
          for (int e = 0; e < E; ++e) acc[h][e] *= w;
        }
      }
      p[h] = ex2(x - (m[h] == -INFINITY ? 0.f : m[h] - 6.f));
      l[h] += part == 0 ? p[h] : 0.f;
    }
    const int t0 = max(0, rq.lo - tok0), t1 = min(8, rq.hi - tok0);   // hidden slots are not read
    const int c = lane * E / 4;
    for (int t = t0; t < t1; ++t) {
      float v[E];
      const uint32_t addr = v_s + (c >> 3) * 1024 + t * 128 + (((c & 7) ^ t) << 4) + (lane * E % 4) * 4;
      if (E == 4) lds4(addr, v);
      else asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(addr));
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float w = __shfl_sync(FULL, p[h], t);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[h][e] = fmaf(w, v[e], acc[h][e]);
      }
    }
  }
  __device__ __forceinline__ static void lds4(uint32_t addr, float* v) {
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(addr));
  }

  template <typename F>
  __device__ __forceinline__ void finish(const DenseArgs& a, bool whole, int lane, F put) {
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float sum = warp_sum(l[h]);
      const float f = whole ? (sum > 0.f ? 1.f / sum : 0.f) : 1.f;
      float* o = put(h, m[h], sum, lane == 0);
#pragma unroll
      for (int e = 0; e < E; ++e) o[lane * E + e] = acc[h][e] * f;
    }
  }
};

template <typename W, int D>
__global__ void __launch_bounds__(DecodeShape<typename W::T, D>::WARPS * 32, 1)
dense_decode_kernel(const __grid_constant__ DecodeMaps maps, const DecodeArgs p) {
  using T = typename W::T;
  using Sh = DecodeShape<T, D>;
  constexpr int TT = Sh::TT, NST = Sh::STAGES, NW = Sh::WARPS;
  constexpr bool F32 = sizeof(T) == 4;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[NW][NST];
  __shared__ int4 s_meta[NW][NST];
  __shared__ __align__(16) float s_q[F32 ? NW : 1][F32 ? 8 * D : 1];
  const DenseArgs& a = p.a;
  const int warp = __shfl_sync(FULL, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int page_shift = a.page_size == 16 ? 4 : 5;
  const uint32_t ring = ((smem_u32(smem_raw) + 1023) & ~1023u) + warp * NST * Sh::STAGE;
  if (lane < NST) mbar_init(&s_bar[warp][lane], 1);
  fence_mbar_init();
  pdl_wait();

  // Tiles of all requests before the run, and the run. A warp looks at 32
  // requests at a time: with no more than that by itself, else the sums of all
  // chunks go through the ring's space, before it is used.
  const int chunks = (a.batch + 31) / 32;
  unsigned* err = blockIdx.x == 0 ? a.err : nullptr;
  auto chunk_tiles = [&](int c, unsigned* e) {         // of the lane's request, all KV heads
    const int r = c * 32 + lane;
    return r < a.batch ? (long long)request_of<TT>(a, r, e).tiles * a.h_kv : 0ll;
  };
  auto running = [&](long long v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(FULL, v, o);
      if (lane >= o) v += t;
    }
    return v;
  };
  long long* sums = reinterpret_cast<long long*>(((uintptr_t)smem_raw + 15) & ~(uintptr_t)15);
  long long n = 0, incl = 0, all;                      // of the lane's request of the chunk in hand
  if (chunks == 1) {
    n = chunk_tiles(0, err);
    incl = running(n);
    all = __shfl_sync(FULL, incl, 31);
  } else {
    for (int c = warp; c < chunks; c += NW) {
      const long long sum = __shfl_sync(FULL, running(chunk_tiles(c, err)), 31);
      if (lane == 0) sums[c] = sum;
    }
    __syncthreads();
    if (warp == 0) {
      long long base = 0;
      for (int c0 = 0; c0 < chunks; c0 += 32) {
        const long long own = c0 + lane < chunks ? sums[c0 + lane] : 0, up = running(own);
        if (c0 + lane < chunks) sums[c0 + lane] = base + up - own;
        base += __shfl_sync(FULL, up, 31);
      }
      if (lane == 0) sums[chunks] = base;
    }
    __syncthreads();
    all = sums[chunks];
  }
  const long long run = run_length(all, p.n_warps);
  // neighbouring runs on different SMs: few tiles spread over the device
  const int wid = warp * gridDim.x + blockIdx.x;
  const long long first = min(all, wid * run), last = min(all, first + run);

  // for the joining kernel: where each request starts (a share per CTA)
  for (int c = blockIdx.x * NW + warp; c < chunks; c += gridDim.x * NW) {
    if (chunks > 1) {
      n = chunk_tiles(c, nullptr);
      incl = running(n);
    }
    if (c * 32 + lane < a.batch) p.starts[c * 32 + lane] = (chunks > 1 ? sums[c] : 0) + incl - n;
    if (c == chunks - 1 && lane == 0) p.starts[a.batch] = all;
  }

  // the run's first request
  int r = 0, g = 0, at = 0;                            // load cursor: request, KV head, tile of it
  Request rq{};
  if (first < last) {
    int c = 0;
    long long base = 0;
    if (chunks > 1) {
      // the last chunk that starts at or before it (chunks without tiles start
      // where the next one does)
      for (int c0 = 0; c0 < chunks; c0 += 32) {
        const unsigned le = __ballot_sync(FULL, c0 + lane < chunks && sums[c0 + lane] <= first);
        if (!le) break;
        c = c0 + 31 - __clz(le);
      }
      base = sums[c];
      n = chunk_tiles(c, nullptr);
      incl = running(n);
    }
    const long long off = first - base;
    const int src = __ffs(__ballot_sync(FULL, off >= incl - n && off < incl)) - 1;
    r = c * 32 + src;
    const long long in = off - __shfl_sync(FULL, incl - n, src);
    rq = request_of<TT>(a, r, nullptr);
    g = (int)(in / rq.tiles);
    at = (int)(in - (long long)g * rq.tiles);
  }
  if (chunks > 1) {
    fence_proxy_async_smem();
    __syncthreads();                                   // sums are read; the ring may fill
  }
  pdl_launch_dependents();
  if (first >= last) return;

  const int total = (int)(last - first);
  const float scale2 = a.scale * LOG2E;
  const uint64_t pol = evict_first_policy();
  int issued = 0;
  int ids = 0, ids_at = -1, ids_r = -1;                // page ids of 32 tiles, one per lane

  const bool fault = a.test_fault == 2 && blockIdx.x == 0 && warp == 0;

  // Start the copies of the cursor's tile into a place of the ring, and step on.
  auto issue = [&](int st) {
    if (ids_r != r || at < ids_at || at >= ids_at + 32) {
      ids_r = r;
      ids_at = at;
      ids = at + lane < rq.tiles ? a.page_indices[rq.e0 + ((rq.tile0 + at + lane) * TT >> page_shift)] : 0;
    }
    const int id = __shfl_sync(FULL, ids, at - ids_at);
    const bool bad = id < 0 || id >= a.n_phys;
    if (lane == 0) {
      s_meta[warp][st] = make_int4(r, g, at, bad);
      if (!bad) {
        uint64_t* bar = &s_bar[warp][st];
        mbar_expect_tx(bar, Sh::STAGE + (fault && st == 0 ? 16 : 0));
        const int y = ((id * a.h_kv + g) << page_shift) + ((rq.tile0 + at) * TT & (a.page_size - 1));
        const uint32_t dst = ring + st * Sh::STAGE;
#pragma unroll
        for (int b = 0; b < Sh::BOXES; ++b) {
          tma_2d_hint(dst + b * Sh::BOX, &maps.k, b * Sh::COLS, y, smem_u32(bar), pol);
          tma_2d_hint(dst + Sh::TILE + b * Sh::BOX, &maps.v, b * Sh::COLS, y, smem_u32(bar), pol);
        }
      } else {
        report(a.err, QUEST_DEVERR_PAGE_RANGE);
      }
    }
    if (++issued < total && ++at == rq.tiles) {
      at = 0;
      if (++g == a.h_kv) {
        g = 0;
        // the next request with a tile, 32 at a time (there is one: more is to come)
        for (int r0 = r + 1;; r0 += 32) {
          const int n = r0 + lane < a.batch ? request_of<TT>(a, r0 + lane, nullptr).tiles : 0;
          const unsigned some = __ballot_sync(FULL, n > 0);
          if (some || r0 + 32 >= a.batch) {
            r = some ? r0 + __ffs(some) - 1 : a.batch - 1;
            break;
          }
        }
        rq = request_of<TT>(a, r, nullptr);
      }
    }
  };

  W w;
  Request cq{};
  int cr = -1, cg = -1, c_first = 0;                   // unit being computed, its first tile here
  auto flush = [&](int next_tile) {
    // the whole unit in this run: write it; a part: to the workspace
    const bool whole = c_first == 0 && next_tile == cq.tiles;
    const size_t row = ((size_t)cr * a.h_kv + cg) * a.group;
    const size_t slot = ((size_t)wid + (size_t)cr * a.h_kv + cg) * a.group;
    w.finish(a, whole, lane, [&](int h, float m, float l, bool mine) {
      if (whole) {
        if (mine && a.lse) a.lse[row + h] = l > 0.f ? (m - 6.f + lg2(l)) * LN2 : -INFINITY;
        return static_cast<float*>(a.out) + (row + h) * D;
      }
      if (mine) p.part_ml[slot + h] = make_float2(m, l);
      return p.part_o + (slot + h) * D;
    });
  };

  for (int k = 0; k < NST && k < total; ++k) issue(k);
  int st = 0, done = 0;
  uint32_t phase = 0;                                  // a bit per place
  bool ok = true;
  int4 meta = make_int4(0, 0, 0, 0);
  for (; done < total; ++done) {
    __syncwarp();
    meta = s_meta[warp][st];
    if (meta.x != cr || meta.y != cg) {
      if (cr >= 0) flush(cq.tiles);
      if (meta.x != cr) cq = request_of<TT>(a, meta.x, nullptr);
      cr = meta.x;
      cg = meta.y;
      c_first = meta.z;
      w.begin(a, cr, cg, lane, s_q[F32 ? warp : 0]);
    }
    if (!meta.w) {
      if (!warp_wait_bounded(&s_bar[warp][st], phase >> st & 1, p.wait_limit)) { ok = false; break; }
      phase ^= 1u << st;
      const uint32_t at_s = ring + st * Sh::STAGE;
      w.tile(a, cq, (cq.tile0 + meta.z) * TT, at_s, at_s + Sh::TILE, s_q[F32 ? warp : 0], scale2, lane);
    }
    __syncwarp();
    if (done + NST < total) issue(st);
    if (++st == NST) st = 0;
  }
  if (!ok) {                                           // report, and wait for the copies in flight
    if (lane == 0) report(a.err, QUEST_DEVERR_WAIT_TIMEOUT);
    for (int k = 0; k < NST && done + k < total; ++k) {
      const int i = (st + k) % NST;
      if (!s_meta[warp][i].w) warp_wait_bounded(&s_bar[warp][i], phase >> i & 1, p.wait_limit);
    }
    return;
  }
  flush(meta.z + 1);
}

// Joins the parts of one (request, query head): the threads take the parts'
// maxima and sums and leave each part's weight in shared memory, then the warps
// every eighth part's o (loads without anything to wait for), whose sums meet
// in shared memory, in a fixed order.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) dense_decode_join_kernel(const DecodeArgs p) {
  constexpr int E = D / 32, CHUNK = 1024;
  __shared__ float s_o[kJoinWarps][D], s_w[CHUNK], s_red[2][kJoinWarps];
  const DenseArgs& a = p.a;
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / a.group, h = blockIdx.x % a.group;
  const int r = unit / a.h_kv, g = unit % a.h_kv;
  const long long run = run_length(p.starts[a.batch], p.n_warps);
  const long long n = (p.starts[r + 1] - p.starts[r]) / a.h_kv, u0 = p.starts[r] + g * n;
  const size_t row = (size_t)unit * a.group + h;
  float* out = static_cast<float*>(a.out) + row * D;
  if (n == 0) {                                        // sees no key
    if (threadIdx.x < D) out[threadIdx.x] = 0.f;
    if (threadIdx.x == 0 && a.lse) a.lse[row] = -INFINITY;
    return;
  }
  const int w0 = (int)(u0 / run), parts = (int)((u0 + n - 1) / run) - w0 + 1;
  if (parts == 1) return;                              // written whole
  const size_t slot0 = ((size_t)w0 + unit) * a.group + h;
  float m = -INFINITY, l = 0.f, o[E] = {};
  for (int c0 = 0; c0 < parts; c0 += CHUNK) {
    const int cnt = min(CHUNK, parts - c0);
    float2 ml[CHUNK / kJoinThreads];
    float mx = m;
#pragma unroll
    for (int k = 0; k < CHUNK / kJoinThreads; ++k) {
      const int i = k * kJoinThreads + threadIdx.x;
      ml[k] = i < cnt ? p.part_ml[slot0 + (size_t)(c0 + i) * a.group] : make_float2(-INFINITY, 0.f);
      mx = fmaxf(mx, ml[k].x);
    }
    mx = warp_max(mx);
    __syncthreads();                                   // the last chunk's weights are used
    if (lane == 0) s_red[0][warp] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) mx = fmaxf(mx, s_red[0][w]);
    if (mx == -INFINITY) continue;                     // parts without a key (whole CTA)
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < CHUNK / kJoinThreads; ++k) {
      const int i = k * kJoinThreads + threadIdx.x;
      const float f = ex2(ml[k].x - mx);
      if (i < cnt) s_w[i] = f;
      sum = fmaf(f, ml[k].y, sum);
    }
    sum = warp_sum(sum);
    if (lane == 0) s_red[1][warp] = sum;
    __syncthreads();
    const float f = ex2(m - mx);
    m = mx;
    l *= f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) l += s_red[1][w];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f;
    const float* src = p.part_o + (slot0 + (size_t)c0 * a.group) * D + lane * E;
#pragma unroll 8
    for (int i = warp; i < cnt; i += kJoinWarps) {
      const float* q = src + (size_t)i * a.group * D;
      float v[E];
      if constexpr (E == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(q);
      else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(q);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(s_w[i], v[e], o[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) v += s_o[w][threadIdx.x];
    out[threadIdx.x] = l > 0.f ? v / l : 0.f;
  }
  if (threadIdx.x == 0 && a.lse) a.lse[row] = l > 0.f ? (m - 6.f + lg2(l)) * LN2 : -INFINITY;
}

}  // namespace quest
