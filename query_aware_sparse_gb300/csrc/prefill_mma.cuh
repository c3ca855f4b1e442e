// Prompt attention on the tensor cores, fp16 (quest_prefill_attn).
//
// Mathematics. For a block of query rows (the tokens of one request times the
// group's heads, head fastest) and one KV head: over blocks of BN keys
//   S = Q K^T;  x = mods(S) in base 2, -inf where a row does not see the key;
//   P = 2^(x - m + 6);  l += sum P;  O += P V
// and O / l at the end. m is a maximum of the row so far, but not taken for
// every block: it stays until a row's weights of a block sum to more than 2^15
// (then m is renewed, O and l rescaled, the block's weights done again). The
// usual block so needs no maximum at all, and no weight passes fp16's 65504;
// the factor 2^6 keeps small weights out of fp16's subnormal range. P is
// rounded to fp16 (half a step, 2^-11 of itself) because the second product
// takes fp16 operands; S, m and l stay in fp32, O for kChainKeys keys in the tensor
// core's accumulator, then in fp32.
//
// Bound. 4 D flops per (row, visible key) on tcgen05 against 2 D bytes per key
// and KV head: tensor bound from a few hundred rows on. The softmax runs one
// exponential per (row, key) next to it.
//
// Shape. TILES row tiles of 128 (one accumulator lane per row). With two tiles
// (256 rows, BN = 128) one tile's softmax runs while the tensor core works on
// the other. With one (few rows; BN = 64) the next block's S is issued before
// the softmax of the last, and two CTAs share an SM. Warps 0-3 (and 4-7) are
// the softmax of a tile, one row per thread; then one warp loads Q and K, one
// issues the products, one loads V, one only frees its registers.
//   shared memory: Q [TILES][D/64][128 rows][64], then a ring of K and V blocks
//     [D/64][BN keys][64] in order K V K V, all rows of 128 bytes with the
//     128-byte swizzle, K and V copied by one TMA box per page and 64 dims;
//   TMEM: S (P takes its place, two fp16 per column) and O, fp32.
// K and V of a block are used by both tiles before their place is refilled.
// Rows of V that hold no valid token are zeroed in shared memory (0 * NaN of a
// stale slot would be NaN); such keys' S is replaced, never added to.
//
// Measured (d 128): a 16384-token prompt of 32 heads 1490 us, 1480 TFLOP/s (the
// GPU at its power cap, 1.6 to 1.8 GHz; cuBLAS sustains 1712); in steady state 2560
// cycles for two tiles and 128 keys, of which the products take 2048. 2048 of
// 65536 tokens, 8 KV heads of 4, 1490 us, capped 2160; 16 requests of four tokens
// over up to 32768, 152 us, 6040 GB/s. d 64: 16384 tokens of 32 heads 1080 us.
// Against 64 bits outputs are 2.6e-4 off (2-norm): 1.9e-4 by their own rounding to
// fp16, 1.8e-4 by that of P and the chains. P as two fp16 numbers, as in dense
// decode, would take three products where there are two.
#pragma once

#include "prefill_common.cuh"

namespace quest {

struct PrefillMaps { CUtensorMap q, k, v, out; };

template <int D, int TILES> struct PrefillShape {
  static constexpr int BN = TILES == 2 ? 128 : 64;
  static constexpr int SBUF = TILES == 2 ? 1 : 2;              // S buffers per tile
  static constexpr int HALVES = D / 64;
  static constexpr uint32_t Q_TILE = 128 * D * 2, BLOCK = BN * D * 2;
  static constexpr int STAGES = TILES == 2 ? (D == 128 ? 5 : 8) : (D == 128 ? 4 : 8);
  static constexpr uint32_t SMEM = 1024 + TILES * Q_TILE + STAGES * BLOCK;
  static constexpr int THREADS = TILES * 128 + 128;    // the last four warps: load, issue, two idle
  static constexpr uint32_t O_COL = TILES * SBUF * BN;         // S buffers first
  static constexpr uint32_t TMEM = O_COL + TILES * D <= 128 ? 128 : O_COL + TILES * D <= 256 ? 256 : 512;
  static constexpr int PER_SM = TILES == 2 ? 1 : 2;
  static constexpr int CHAIN = kChainKeys / BN;        // steps
  static_assert((CHAIN & (CHAIN - 1)) == 0, "steps are masked");
};

// x -> 4 tanh(t / 4), t = x * to_t: t is four times the logit over its cap. The error
// goes with the value, not with the cap, as far as a weight can feel it. By the
// largest |t| of a warp's rows:
//   below 2, below 4: t (1 + w R(w)), w = t^2, to 2 units of 2^-24 of the result;
//   caps up to kSmallCap: 4 - 8 / (1 + e^(t / 2)), off by 2^-19 at most: 2^-21 of the
//     cap, 2^-15 in a logit, little next to the rounding of the weights (2^-11);
//   larger caps: t N(w) / D(w), all coefficients positive, to 12 units of the
//     result, |t| held at 32, where tanh is 1 to 4 units: the small logits of rows
//     next to ones near a large cap keep their accuracy.
// R, N and D fitted at Chebyshev nodes. 2048 tokens over 65536 keys, 32 heads, d 128:
// 2.10, 2.88, 3.12 and 3.65 ms. Blocks where a row's keys begin or end (`edge`) take
// one of the last two, value by value the same whatever hidden columns hold; rows
// that are not `live` have no say.
constexpr float kSmallCap = 64.f;
template <int N>
__device__ __forceinline__ void four_tanh(float (&x)[N], float to_t, bool small, bool live, bool edge) {
  float most = 0.f;
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const float2 t = mul2(make_float2(x[c], x[c + 1]), both(to_t));
    x[c] = t.x;
    x[c + 1] = t.y;
    most = fmaxf(fmaxf(most, fabsf(t.x)), fabsf(t.y));
  }
  if (!edge && __all_sync(FULL, most < 2.f || !live)) {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const float2 t = make_float2(x[c], x[c + 1]), w = mul2(t, t);
      float2 v = fma2(w, both(2.744864673331904e-07f), both(-1.3033962204644922e-05f));
      v = fma2(v, w, both(0.0005207217182032764f));
      v = fma2(v, w, both(-0.020833319053053856f));
      v = fma2(v, w, both(1.f));
      v = mul2(v, t);
      x[c] = v.x;
      x[c + 1] = v.y;
    }
  } else if (!edge && __all_sync(FULL, most < 4.f || !live)) {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const float2 t = make_float2(x[c], x[c + 1]), w = mul2(t, t);
      float2 v = fma2(w, both(-1.5672128308649724e-12f), both(1.4963504046949794e-10f));
      v = fma2(v, w, both(-7.838174553853605e-09f));
      v = fma2(v, w, both(3.3050713454940706e-07f));
      v = fma2(v, w, both(-1.3167673387215473e-05f));
      v = fma2(v, w, both(0.0005208253278397024f));
      v = fma2(v, w, both(-0.0208333320915699f));
      v = fma2(v, w, both(1.f));
      v = mul2(v, t);
      x[c] = v.x;
      x[c + 1] = v.y;
    }
  } else if (small) {
#pragma unroll
    for (int c = 0; c < N; ++c) x[c] = fmaf(rcp(1.f + ex2(x[c] * (0.5f * LOG2E))), -8.f, 4.f);
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const float2 t = make_float2(clamp_nan(x[c], 32.f), clamp_nan(x[c + 1], 32.f)), w = mul2(t, t);
      float2 n = fma2(w, both(2.80596501589514e-09f), both(1.1560538951016497e-05f));
      n = fma2(n, w, both(0.008084234781563282f));
      n = fma2(n, w, both(1.f));
      float2 d = fma2(w, both(3.777043348224263e-12f), both(5.8521202106476267e-08f));
      d = fma2(d, w, both(9.317861258750781e-05f));
      d = fma2(d, w, both(0.028917556628584862f));
      d = fma2(d, w, both(1.f));
      n = mul2(mul2(n, t), make_float2(rcp(d.x), rcp(d.y)));
      x[c] = n.x;
      x[c + 1] = n.y;
    }
  }
}

// A warp's sums of finished chains, O of its rows in terms of the maximum was[row],
// kept in the workspace while a new chain runs: rows of D floats, G heads of a token
// side by side, hq rows from token to token, the first of the tile at kept. Adds
// what is kept (`add`) to O and leaves the sum there (`back`) or in O's stead in the
// workspace. Where all 32 rows are live, eight rows' pieces of 32 columns change
// places, so that a warp touches whole lines. Not inlined: it would cost the loop
// around it registers.
template <int D>
__device__ __noinline__ void chain_sums(uint32_t o_col, float* kept, float* kept_m, int hq, int G, int row, float m,
                                        bool live, bool add, bool back) {
  const int shift = __ffs(G) - 1;
  const bool full = __all_sync(FULL, live);
  const float was = add && live ? *kept_m : -INFINITY, f = was == -INFINITY ? 0.f : ex2(was - m);
  auto piece = [&](int c, int e) {
    const int r = full ? (row & ~7) + e : row, i = full ? row & 7 : e;
    return reinterpret_cast<float4*>(kept + ((size_t)(r >> shift) * hq + (r & (G - 1))) * D + c * 32) + i;
  };
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    tmem_ld32(o_col + c * 32, o);
    tmem_wait_ld();
    tmem_loaded(o);
    if (add && live) {
      float4 v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = *piece(c, e);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[4 * e] = __float_as_uint(fmaf(f, v[e].x, __uint_as_float(o[4 * e])));
        o[4 * e + 1] = __float_as_uint(fmaf(f, v[e].y, __uint_as_float(o[4 * e + 1])));
        o[4 * e + 2] = __float_as_uint(fmaf(f, v[e].z, __uint_as_float(o[4 * e + 2])));
        o[4 * e + 3] = __float_as_uint(fmaf(f, v[e].w, __uint_as_float(o[4 * e + 3])));
      }
    }
    __syncwarp();
    if (back) {
      tmem_st32(o_col + c * 32, o);
    } else if (live) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        *piece(c, e) = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                   __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
    }
    __syncwarp();
  }
  if (back) tmem_wait_st();
  else if (live) *kept_m = m;
}

template <int D, int TILES, bool CAP, bool ALIBI>
__global__ void __launch_bounds__(PrefillShape<D, TILES>::THREADS, PrefillShape<D, TILES>::PER_SM)
prefill_mma_kernel(const __grid_constant__ PrefillMaps maps, const PrefillArgs p) {
  using P = PrefillShape<D, TILES>;
  constexpr int BN = P::BN, SBUF = P::SBUF, HALVES = P::HALVES, STAGES = P::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_full, full[STAGES], empty[STAGES], aux, drain;
  __shared__ __align__(8) uint64_t s_full[TILES][SBUF], p_full[TILES][SBUF], pv_done[TILES], o_full[TILES];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_quit, s_bad;

  const DenseArgs& a = p.a;
  const int warp = __shfl_sync(FULL, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int G = a.group, S = a.page_size, hq = a.h_kv * G;
  const int page_shift = S == 16 ? 4 : 5;
  const int tile_tokens = 128 / G;
  int g, split, idx;
  p.place(blockIdx.x, a.h_kv, &g, &split, &idx);

  // Every warp finds the row block and its keys by itself: nothing to wait for
  // until the first copies are on their way.
  int r = 0, blk = 0;
  if (!find_block(a, TILES * tile_tokens, idx, lane, &r, &blk)) return;   // past the last one
  const int row0 = a.q_indptr[r], n_r = a.q_indptr[r + 1] - row0;
  const int e0 = a.page_indptr[r], len = a.seq_lens[r];
  const int held = held_tokens(len, a.page_indptr[r + 1] - e0, S, threadIdx.x ? nullptr : a.err);
  const int prefix = a.prefix_lens ? a.prefix_lens[r] : 0;
  const int tok0 = blk * TILES * tile_tokens;          // first token of the row block

  // key blocks of each tile and of all: from the least that its first row may
  // see to the most its last may (both grow with the position)
  int t0[TILES], t1[TILES], n0 = 0x7fffffff, n1 = 0;
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    const int ta = tok0 + t * tile_tokens, tb = min(min(n_r, a.n_q - row0), ta + tile_tokens);
    int doc = 0x7fffffff;
    if (a.doc_starts) {
      for (int i = ta + lane; i < tb; i += 32) doc = min(doc, a.doc_starts[row0 + i]);
      doc = __reduce_min_sync(FULL, doc);
    } else {
      doc = 0;
    }
    const int lo = seen_keys(len - n_r + ta, held, a.window, doc, prefix).lo;
    const int hi = seen_keys(len - n_r + tb - 1, held, 0, 0, prefix).hi;
    const bool any = ta < tb && hi > lo;
    t0[t] = any ? lo / BN : 0;
    t1[t] = any ? (hi + BN - 1) / BN : 0;
    if (any) {
      n0 = min(n0, t0[t]);
      n1 = max(n1, t1[t]);
    }
  }
  if (n1 == 0) n0 = 0;
  if (p.splits > 1) {
    const int nb = n1 - n0, first = n0;
    n0 = first + (int)((long long)nb * split / p.splits);
    n1 = first + (int)((long long)nb * (split + 1) / p.splits);
  }
  // Blocks are taken from the last key on: step i is key block n1 - 1 - i. Near
  // keys come first, where a distance bias leaves the largest logits, so the
  // maximum seldom has to be renewed (packed documents with a bias: 63 -> 53 us).
  const int nb = n1 - n0;
#pragma unroll
  for (int t = 0; t < TILES; ++t) {                    // each tile's steps
    const int from = max(n0, t0[t]), to = min(n1, t1[t]);
    t0[t] = n1 - to;
    t1[t] = n1 - from;
  }
  const bool softmax_warp = warp < 4 * TILES;
  const uint32_t q_s = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t ring = q_s + TILES * P::Q_TILE;
  const int pages_per_block = BN / S;

  // A step's pages into their place of the ring: the lanes' page ids, then a box
  // per page and 64 dims
  auto page_of = [&](int i) {
    const int lp = (n1 - 1 - i) * pages_per_block + lane;
    int id = -1;
    if (lane < pages_per_block && i < nb && lp << page_shift < held) id = a.page_indices[e0 + lp];
    return id >= 0 && id < a.n_phys ? id : -1;
  };
  auto copy = [&](const CUtensorMap* map, int id, uint32_t dst, uint64_t* bar, uint32_t bytes) {
    if (lane == 0 && bytes) mbar_expect_tx(bar, bytes);
    __syncwarp();
    if (id >= 0) {
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
        tma_2d(dst + h * BN * 128 + lane * S * 128, map, h * 64, (id * a.h_kv + g) * S, smem_u32(bar));
    }
    __syncwarp();
  };
  auto block_bytes = [&](int id) { return __popc(__ballot_sync(FULL, id >= 0)) * S * D * 2u; };

  int id = -1;                                         // the loaders' page of the next block
  if (warp == 4 * TILES) {
    if (lane == 0) {
      mbar_init(&q_full, 1);
      mbar_init(&aux, 1);
      mbar_init(&drain, 1);
      for (int i = 0; i < STAGES; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
      for (int t = 0; t < TILES; ++t) {
        for (int i = 0; i < SBUF; ++i) { mbar_init(&s_full[t][i], 1); mbar_init(&p_full[t][i], 4); }
        mbar_init(&pv_done[t], 1);
        mbar_init(&o_full[t], 1);
      }
      fence_mbar_init();
      s_quit = 0;
      s_bad = 0;
      if (nb > 0) {
        mbar_expect_tx(&q_full, TILES * P::Q_TILE);
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
            tma_3d(q_s + t * P::Q_TILE + h * 128 * 128, &maps.q, h * 64, g * G,
                   row0 + tok0 + t * tile_tokens, smem_u32(&q_full));
      }
    }
    __syncwarp();
    if (nb > 0) {
      id = page_of(0);
      const uint32_t bytes = block_bytes(id);
      if (a.test_fault == 2 && blockIdx.x == 0 && lane == 0) mbar_expect_more(&full[0], 16);
      copy(&maps.k, id, ring, &full[0], bytes);
      if (lane == 0 && !bytes) mbar_arrive(&full[0]);
      id = page_of(1);
    }
  } else if (warp == 4 * TILES + 1) {
    tmem_alloc(smem_u32(&s_tmem), P::TMEM);
  } else if (warp == 4 * TILES + 2) {
    id = page_of(0);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // two tiles: 384 threads of 168 registers, 256 x 208 + 128 x 80 = 63488 of 64512
  if (warp == 4 * TILES || warp == 4 * TILES + 2) {
    // ---- loads: one warp the K blocks and Q, another the V blocks ---------------
    if (TILES == 2) regs_down<80>();
    const int kv = warp == 4 * TILES ? 0 : 1;
    uint32_t aux_phase = 0;
    bool go = true;
    int seq = 2 - kv;                                  // block seq of the ring's sequence
    for (int i = 1 - kv; i < nb; ++i, seq += 2) {
      const int next = page_of(i + 1), n = n1 - 1 - i;
      const unsigned have = __ballot_sync(FULL, id >= 0);
      const uint32_t bytes = block_bytes(id);
      const bool ragged = held < (n + 1) * BN || __popc(have) < pages_per_block;
      const int stage = seq % STAGES;
      if (seq >= STAGES &&
          !(go = warp_wait_or_quit(&empty[stage], (seq / STAGES & 1) ^ 1, p.wait_limit, &s_quit)))
        break;
      const uint32_t dst = ring + stage * P::BLOCK;
      copy(kv ? &maps.v : &maps.k, id, dst, kv && ragged ? &aux : &full[stage], bytes);
      if (kv && ragged) {
        // zero what is no valid token, then hand the block over
        if (bytes) {
          if (!(go = warp_wait_or_quit(&aux, aux_phase, p.wait_limit, &s_quit))) break;
          aux_phase ^= 1;
        }
        for (int c = lane; c < BN * HALVES * 8; c += 32) {
          const int row = c >> 3 & (BN - 1), h = c / (8 * BN);
          if (n * BN + row >= held || !(have >> (row >> page_shift) & 1)) {
            const uint32_t at = dst + h * BN * 128 + row * 128 + (c & 7) * 16;
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" :: "r"(at), "r"(0) : "memory");
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[stage]);
      } else if (!bytes && lane == 0) {
        mbar_arrive(&full[stage]);
      }
      id = next;
    }
    if (s_quit) {                                      // wait (bounded) for the copies in flight
      for (int k = seq - 2; k >= 0 && k > seq - 2 - STAGES; k -= 2)
        for (uint32_t i = 0; i < p.wait_limit && !mbar_try_wait_sleep(&full[k % STAGES], k / STAGES & 1, 1000u); ++i) {}
      for (uint32_t i = 0; i < p.wait_limit && kv == 0 && nb > 0 && !mbar_try_wait_sleep(&q_full, 0, 1000u); ++i) {}
    }
  } else if (warp == 4 * TILES + 1) {
    // ---- tensor core: the warp stays converged, one lane issues ------------------
    if (TILES == 2) regs_down<80>();
    const int blocks = __shfl_sync(FULL, nb, 0);
    // the steps in which the tiles take part
    const int a0 = __shfl_sync(FULL, t0[0], 0), b0 = __shfl_sync(FULL, t1[0], 0);
    const int a1 = __shfl_sync(FULL, t0[TILES - 1], 0), b1 = __shfl_sync(FULL, t1[TILES - 1], 0);
    const uint32_t tm = __shfl_sync(FULL, tmem, 0);
    const uint32_t lead = elect_one();
    if (blocks > 0) {
      constexpr uint32_t ID_S = mma_idesc(128, BN, false), ID_O = mma_idesc(128, D, true);
      const uint64_t q_d = smem_desc(q_s, 16, 1024), k_d = smem_desc(ring, 16, 1024);
      const uint64_t v_d = smem_desc(ring, BN * 128, 1024);
      const int chain = p.chained ? P::CHAIN - 1 : -1;
      auto active = [&](int t, int n) { return t == 0 ? n >= a0 && n < b0 : n >= a1 && n < b1; };
      auto issue_s = [&](int t, int buf, int stage) {
        const uint64_t qd = q_d + t * (P::Q_TILE >> 4), kd = k_d + stage * (P::BLOCK >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(lead, tm + (t * SBUF + buf) * BN, qd + ((k >> 2) * 128 * 128 + (k & 3) * 32 >> 4),
                 kd + ((k >> 2) * BN * 128 + (k & 3) * 32 >> 4), ID_S, k > 0);
        mma_commit(lead, &s_full[t][buf]);
      };
      auto issue_o = [&](int t, int buf, int stage, bool acc) {
        const uint64_t vd = v_d + stage * (P::BLOCK >> 4);
#pragma unroll
        for (int k = 0; k < BN / 16; ++k)
          mma_ts(lead, tm + P::O_COL + t * D, tm + (t * SBUF + buf) * BN + k * 8, vd + (k * 2048 >> 4),
                 ID_O, acc || k > 0);
      };
      // places of the ring: K of block n, then V of it, then K of block n + 1
      int ks = 0, vs = 1;
      uint32_t kp = 0, vp = 0, p_phase = 0;           // their phases; a bit per S buffer
      auto k_next = [&]() { ks += 2; if (ks >= STAGES) { ks -= STAGES; kp ^= 1; } };
      auto v_next = [&]() { vs += 2; if (vs >= STAGES) { vs -= STAGES; vp ^= 1; } };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = warp_wait_or_quit(bar, parity, p.wait_limit, &s_quit);
        tc_fence_after();
        return ok;
      };
      bool go = wait(&q_full, 0) && wait(&full[0], 0);
      if (go) {
#pragma unroll
        for (int t = 0; t < TILES; ++t)
          if (active(t, 0)) issue_s(t, 0, 0);
        mma_commit(lead, &empty[0]);
        k_next();
      }
      for (int n = 0; go && n < blocks; ++n) {
        const int buf = SBUF == 2 ? n & 1 : 0;
        const bool more = n + 1 < blocks;
        if (SBUF == 2 && more) {                      // the next S while this softmax runs
          if (!(go = wait(&full[ks], kp))) break;
          if (active(0, n + 1)) issue_s(0, buf ^ 1, ks);
          mma_commit(lead, &empty[ks]);
          k_next();
        }
        if (!(go = wait(&full[vs], vp))) break;
        if (SBUF == 1 && more && !(go = wait(&full[ks], kp))) break;
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          if (active(t, n)) {
            const int bit = t * SBUF + buf;
            if (!(go = wait(&p_full[t][buf], p_phase >> bit & 1))) break;
            p_phase ^= 1u << bit;
            issue_o(t, buf, vs, ((n - (t == 0 ? a0 : a1)) & chain) != 0);   // a new chain: O = P V
            if (SBUF == 2) mma_commit(lead, &pv_done[t]);
            if (n + 1 == (t == 0 ? b0 : b1)) mma_commit(lead, &o_full[t]);
          }
          if (t == TILES - 1) mma_commit(lead, &empty[vs]);
          if (SBUF == 1 && more) {
            if (active(t, n + 1)) issue_s(t, 0, ks);
            if (t == TILES - 1) mma_commit(lead, &empty[ks]);
          }
        }
        if (SBUF == 1 && more) k_next();
        v_next();
      }
      // everything issued is done before the CTA may leave (bounded)
      mma_commit(lead, &drain);
      for (uint32_t k = 0; k < p.wait_limit && !mbar_try_wait_sleep(&drain, 0, 1000u); ++k) {}
    }
  } else if (softmax_warp) {
    // ---- softmax: one row per thread ------------------------------------------------
    if (TILES == 2) regs_up<208>();
    const int tile = warp >> 2, row = threadIdx.x & 127;
    const int tok = tok0 + tile * tile_tokens + row / G, pos = len - n_r + tok;
    const bool valid = tok < n_r && row0 + tok < a.n_q;
    Seen seen{0, 0};
    if (valid) seen = seen_keys(pos, held, a.window, a.doc_starts ? a.doc_starts[row0 + tok] : 0, prefix);
    // A row that sees nothing, or is none, is not looked at: its weights may be
    // anything, they reach no other row, and its l is taken as 0 at the end.
    const bool live = seen.hi > seen.lo;
    // pages outside the pool: reported, and looked for block by block if any
    for (int pg = (n0 * BN >> page_shift) + (int)threadIdx.x; pg < min(n1 * BN, held + S - 1) >> page_shift;
         pg += TILES * 128) {
      const int page = a.page_indices[e0 + pg];
      if (page < 0 || page >= a.n_phys) s_bad = 1;
    }
    bar_sync<1, TILES * 128>();
    const bool any_bad = s_bad != 0;
    if (any_bad && threadIdx.x == 0) report(a.err, QUEST_DEVERR_PAGE_RANGE);
    const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
    const int h = g * G + row % G;
    const float log2s = a.scale * LOG2E;
    const float cap2_4 = 0.25f * a.softcap * LOG2E, to_t = CAP ? 4.f * a.scale / a.softcap : 0.f;
    const float slope2 = ALIBI && valid ? a.slopes[h] * LOG2E : 0.f;
    const float sl2 = ALIBI ? 1.f : CAP ? cap2_4 : log2s;   // of the value the maximum is taken of
    float m = live ? -INFINITY : 0.f, l = 0.f;
    uint32_t s_phase = 0;                             // a bit per S buffer
    bool ok = true;
    const int first = tile == 0 ? t0[0] : t0[TILES - 1], last = tile == 0 ? t1[0] : t1[TILES - 1];
    const uint32_t o_col = tmem + lanes + P::O_COL + tile * D;
    // sums of finished chains: the tile's rows, this row's maximum
    float* kept = p.part_o + (((size_t)split * a.n_q + row0 + tok0 + tile * tile_tokens) * hq + g * G) * D;
    float* kept_m = p.part_lse + ((size_t)split * a.n_q + row0 + tok) * hq + h;
    for (int from = first, to; from < last; from = to) {   // chain by chain
      to = p.chained ? min(last, from + P::CHAIN) : last;
      for (int i = from; i < to; ++i) {
        const int buf = SBUF == 2 ? i & 1 : 0, n = n1 - 1 - i;
        const uint32_t s_col = tmem + lanes + (tile * SBUF + buf) * BN;
        unsigned bad = 0;
        if (any_bad) {
          const int lp = n * pages_per_block + lane;
          const int page = lane < pages_per_block && lp << page_shift < held ? a.page_indices[e0 + lp] : 0;
          bad = __ballot_sync(FULL, page < 0 || page >= a.n_phys);
        }
        if (!(ok = warp_wait_or_quit(&s_full[tile][buf], s_phase >> buf & 1, p.wait_limit, &s_quit))) break;
        s_phase ^= 1u << buf;
        tc_fence_after();
        uint32_t sv[BN / 32][32];
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) tmem_ld32(s_col + c * 32, sv[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) tmem_loaded(sv[c]);
        float x[BN];
#pragma unroll
        for (int c = 0; c < BN; ++c) x[c] = __uint_as_float(sv[c / 32][c % 32]);
        const int kb = n * BN;
        const bool edge = __any_sync(FULL, live && (kb < seen.lo || kb + BN > seen.hi || bad));
        auto hidden = [&](int c) { return kb + c < seen.lo || kb + c >= seen.hi || (bad >> (c >> page_shift) & 1); };
        if (CAP) four_tanh<BN>(x, to_t, a.softcap <= kSmallCap, live, edge);
        if (ALIBI) {
          const float d0 = (float)(pos - kb);
#pragma unroll
          for (int c = 0; c < BN; ++c)
            x[c] = fmaf(fabsf(d0 - (float)c), -slope2, x[c] * (CAP ? cap2_4 : log2s));
        }
        if (edge) {
#pragma unroll
          for (int c = 0; c < BN; ++c)
            if (hidden(c)) x[c] = -INFINITY;
        }
        // The maximum lags: with it the block's weights, and only where their sum
        // passes 2^15 (one above 2^14 is among them, or many above 2^8) or a row
        // has no maximum yet is a new one taken and the weights done again.
        float sum;
        bool again = __any_sync(FULL, m == -INFINITY);
        for (bool once = false;; once = true) {
          if (again) {
            float mc[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int c = 4; c < BN; c += 4)
#pragma unroll
              for (int e = 0; e < 4; ++e) mc[e] = fmaxf(mc[e], x[c + e]);
            const float mx = fmaxf(m, fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3])) * sl2);
            const float f = mx > m ? ex2(m - mx) : 1.f;   // m = -inf: O and l are zero, f = 0
            m = mx;
            l *= f;
            if (i > from) {
              // the products up to step i - 1 are in O: with one S buffer the S
              // that was waited for came after them, with two it came after i - 2
              if (SBUF == 2 && !(ok = warp_wait_or_quit(&pv_done[tile], (i - 1 - first) & 1, p.wait_limit, &s_quit)))
                break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(o_col + c * 32, o);
                tmem_wait_ld();
                tmem_loaded(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(o_col + c * 32, o);
              }
            }
          }
          const float mu = m == -INFINITY ? 0.f : m - 6.f;
          float2 sums[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 sl = make_float2(sl2, sl2), nmu = make_float2(-mu, -mu);
#pragma unroll
          for (int c = 0; c < BN / 64; ++c) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float2 v = make_float2(x[c * 64 + 2 * e], x[c * 64 + 2 * e + 1]);
              v = fma2(v, sl, nmu);
              v = make_float2(ex2(v.x), ex2(v.y));
              sums[e & 1] = add2(sums[e & 1], v);
              const __half2 hh = __floats2half2_rn(v.x, v.y);
              w[e] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            tmem_st32(s_col + c * 32, w);
          }
          sum = (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
          if (once) break;
          again = __any_sync(FULL, live && sum > 32768.f);
          if (!again) break;
        }
        if (!ok) break;
        l += sum;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[tile][buf]);
      }
      if (!ok || to == last) break;
      // The chain's sums leave O, which the next step's product begins anew. The next
      // S being there, the products up to the last step but one are done, and with
      // one S buffer the last; with two that has its own barrier, whose phase can be
      // told now.
      const int buf = SBUF == 2 ? to & 1 : 0;
      if (!(ok = warp_wait_or_quit(&s_full[tile][buf], s_phase >> buf & 1, p.wait_limit, &s_quit))) break;
      if (SBUF == 2 && !(ok = warp_wait_or_quit(&pv_done[tile], (to - 1 - first) & 1, p.wait_limit, &s_quit)))
        break;
      tc_fence_after();
      chain_sums<D>(o_col, kept, kept_m, hq, G, row, m, live, from > first, false);
    }
    // A full tile goes through the place of its queries (read by now: the
    // products are done) to one TMA store; another row by row.
    const bool whole = p.splits == 1 && last > first && tok0 + (tile + 1) * tile_tokens <= n_r;
    const uint32_t q_at = q_s + tile * P::Q_TILE;
    // ---- O / l ------------------------------------------------------------------------
    if (ok && last > first)
      ok = warp_wait_or_quit(&o_full[tile], 0, p.wait_limit, &s_quit);
    if (ok) {
      tc_fence_after();
      if (p.chained && last - first > P::CHAIN) chain_sums<D>(o_col, kept, kept_m, hq, G, row, m, live, true, true);
      const bool some = live && l > 0.f;               // has a key
      const float inv = some ? 1.f / l : 0.f;
      const float lse2 = some ? m - 6.f + lg2(l) : -INFINITY;
      const size_t at = ((size_t)row0 + tok) * hq + h, part = (size_t)split * a.n_q * hq + at;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (last > first) {
          tmem_ld32(o_col + c * 32, o);
          tmem_wait_ld();
          tmem_loaded(o);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e)
          o[e] = some ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
        if (p.splits > 1) {
          float* dst = p.part_o + part * D + c * 32;
          if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) st_v8(dst + e, o + e);
          }
        } else {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const __half2 hh = __floats2half2_rn(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
            w[e] = *reinterpret_cast<const uint32_t*>(&hh);
          }
          if (whole) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};"
                           :: "r"(q_at + (c >> 1) * 128 * 128 + row * 128 + ((((c & 1) * 4 + e) ^ (row & 7)) << 4)),
                              "r"(w[4 * e]), "r"(w[4 * e + 1]), "r"(w[4 * e + 2]), "r"(w[4 * e + 3]) : "memory");
          } else if (valid) {
            __half* dst = static_cast<__half*>(a.out) + at * D + c * 32;
#pragma unroll
            for (int e = 0; e < 16; e += 8) st_v8(dst + 2 * e, w + e);
          }
        }
        __syncwarp();
      }
      if (valid) {
        if (p.splits > 1) p.part_lse[part] = lse2;
        else if (a.lse) a.lse[at] = lse2 * LN2;
      }
    }
    if (whole) {                                       // the tile's four warps, also after a wait ran out
      fence_proxy_async_smem();
      if (tile == 0) bar_sync<2, 128>();
      else bar_sync<3, 128>();
      if (row == 0 && !s_quit) {
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
          tma_store_3d(&maps.out, q_at + hf * 128 * 128, hf * 64, g * G, row0 + tok0 + tile * tile_tokens);
        tma_store_wait();
      }
    }
  } else if (TILES == 2) {
    regs_down<80>();
  }
  tc_fence_before();
  __syncthreads();
  if (s_quit && threadIdx.x == 0) report(a.err, QUEST_DEVERR_WAIT_TIMEOUT);
  if (warp == 4 * TILES + 1) tmem_free(tmem, P::TMEM);
}

template <int D, int TILES>
cudaError_t launch_prefill_mma_t(const PrefillMaps& maps, const PrefillArgs& p, cudaStream_t s) {
  using P = PrefillShape<D, TILES>;
  const unsigned grid = (unsigned)p.blocks * p.a.h_kv * p.splits;
  auto go = [&](auto kernel) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, P::SMEM);
    if (e != cudaSuccess) return e;
    kernel<<<grid, P::THREADS, P::SMEM, s>>>(maps, p);
    return cudaGetLastError();
  };
  const bool cap = p.a.softcap > 0.f, alibi = p.a.slopes != nullptr;
  cudaError_t e = cap ? (alibi ? go(prefill_mma_kernel<D, TILES, true, true>)
                               : go(prefill_mma_kernel<D, TILES, true, false>))
                      : (alibi ? go(prefill_mma_kernel<D, TILES, false, true>)
                               : go(prefill_mma_kernel<D, TILES, false, false>));
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_prefill_join<__half, D>(p, s);
}

}  // namespace quest
