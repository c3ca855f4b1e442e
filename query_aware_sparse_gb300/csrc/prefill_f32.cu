// Prompt attention, fp32 (quest_prefill_attn): the same sums on plain FMA, all
// of it in fp32.
//
// A CTA of 256 threads takes 128 rows (tokens times the group's heads) and 64
// keys at a time from shared memory; a thread 8 rows x 4 keys of S (its keys
// 16 apart, so that rows padded by 16 bytes are read without bank conflicts),
// then 8 rows x D / 16 dims of O from P (transposed) and V. FMA bound, if the
// tile is this large: 12 16-byte shared loads per 128 FMA for S (with 4 x 4 keys
// 8 per 64, twice what shared memory delivers; 27 -> 31 TFLOP/s at d 64, 36 at 128), 4 per
// 64 for O. The next block's K and V come by cp.async meanwhile.
#include "prefill_common.cuh"

namespace quest {
namespace {

constexpr int kRows = 128, kKeys = 64, kR = kRows / 16;   // rows of a CTA and of a thread

template <int D> struct ShapeF32 {
  static constexpr int LD = D + 4, LP = kRows + 4;
  static constexpr int STAGE = 2 * kKeys * LD;         // floats: K, V
  static constexpr bool P_OVER_K = LP <= LD;           // P takes K's place once S is there
  static constexpr int SMEM = (kRows * LD + 2 * STAGE + (P_OVER_K ? 0 : kKeys * LP)) * (int)sizeof(float);
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               :: "r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}

template <int D>
__global__ void __launch_bounds__(256, 1) prefill_f32_kernel(const PrefillArgs p) {
  using Sh = ShapeF32<D>;
  constexpr int LD = Sh::LD, LP = Sh::LP, C4 = D / 4, OC = D / 64;
  extern __shared__ __align__(16) float smem[];
  float* s_q = smem;
  float* s_kv = s_q + kRows * LD;                      // two stages of K, V
  __shared__ int s_req, s_blk, s_lo, s_hi;
  const DenseArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, tx = tid & 15, ty = tid >> 4;
  const int G = a.group, S = a.page_size, hq = a.h_kv * G, tokens = kRows / G;

  int g, split, idx;
  p.place(blockIdx.x, a.h_kv, &g, &split, &idx);
  if (tid < 32) {
    int r = -1, blk = 0;
    const bool found = find_block(a, tokens, idx, lane, &r, &blk);
    if (lane == 0) { s_req = found ? r : -1; s_blk = blk; s_lo = 0x7fffffff; s_hi = 0; }
  }
  __syncthreads();
  const int r = s_req;
  if (r < 0) return;
  const int row0 = a.q_indptr[r], n_r = a.q_indptr[r + 1] - row0;
  const int e0 = a.page_indptr[r], len = a.seq_lens[r];
  const int held = held_tokens(len, a.page_indptr[r + 1] - e0, S, tid ? nullptr : a.err);
  const int tok0 = s_blk * tokens;

  Seen seen[kR];
  int pos[kR];
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int tok = tok0 + (ty * kR + i) / G;
    pos[i] = len - n_r + tok;
    seen[i] = Seen{0, 0};
    if (tok < n_r && row0 + tok < a.n_q)
      seen[i] = seen_keys(pos[i], held, a.window, a.doc_starts ? a.doc_starts[row0 + tok] : 0,
                          a.prefix_lens ? a.prefix_lens[r] : 0);
    if (seen[i].hi <= seen[i].lo) seen[i] = Seen{0, 0};
    if (tx == 0 && seen[i].hi > 0) {
      atomicMin(&s_lo, seen[i].lo);
      atomicMax(&s_hi, seen[i].hi);
    }
  }
  for (int i = tid; i < kRows * C4; i += 256) {
    const int row = i / C4, c = i % C4, tok = tok0 + row / G;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (tok < n_r && row0 + tok < a.n_q)
      v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                           ((size_t)(row0 + tok) * hq + g * G + row % G) * D + c * 4);
    *reinterpret_cast<float4*>(s_q + row * LD + c * 4) = v;
  }
  __syncthreads();
  int n0 = s_hi > 0 ? s_lo / kKeys : 0, n1 = (s_hi + kKeys - 1) / kKeys;
  const int nb = n1 - n0, first = n0;
  n0 = first + (int)((long long)nb * split / p.splits);
  n1 = first + (int)((long long)nb * (split + 1) / p.splits);

  const float log2s = a.scale * LOG2E, cap2 = a.softcap * LOG2E, inv_cap2 = 1.f / cap2;
  float slope2[kR], m[kR], l[kR], o[kR][OC][4];
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    slope2[i] = a.slopes ? a.slopes[g * G + (ty * kR + i) % G] * LOG2E : 0.f;
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < OC; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][c][e] = 0.f;
  }

  // K and V rows of block n into its stage; zeros where there is no token
  auto fetch = [&](int n) {
    float* s_k = s_kv + (n & 1) * Sh::STAGE;
    float* s_v = s_k + kKeys * LD;
#pragma unroll 4
    for (int i = tid; i < kKeys * C4; i += 256) {
      const int row = i / C4, c = i % C4, j = n * kKeys + row;
      const int id = n < n1 && j < held ? a.page_indices[e0 + j / S] : -1;
      const bool there = id >= 0 && id < a.n_phys;
      const size_t at = there ? (((size_t)id * a.h_kv + g) * S + j % S) * D + c * 4 : 0;
      cp_async16(s_k + row * LD + c * 4, static_cast<const float*>(a.k_pool) + at, there);
      cp_async16(s_v + row * LD + c * 4, static_cast<const float*>(a.v_pool) + at, there);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (n0 < n1) fetch(n0);
  for (int n = n0; n < n1; ++n) {
    const int kb = n * kKeys;
    const float* s_k = s_kv + (n & 1) * Sh::STAGE;
    const float* s_v = s_k + kKeys * LD;
    float* s_p = Sh::P_OVER_K ? s_kv + (n & 1) * Sh::STAGE : s_kv + 2 * Sh::STAGE;   // [key][row]
    fetch(n + 1);
    unsigned long long bad = 0;                        // keys of pages outside the pool
    for (int q = 0; q < kKeys / S; ++q) {
      if (kb + q * S >= held) break;
      const int id = a.page_indices[e0 + kb / S + q];
      if (id < 0 || id >= a.n_phys) {
        bad |= ((1ull << S) - 1) << (q * S);
        if (tid == 0) report(a.err, QUEST_DEVERR_PAGE_RANGE);
      }
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();

    float s[kR][4];
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 2
    for (int c = 0; c < C4; ++c) {
      float4 k[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4*>(s_k + (tx + 16 * j) * LD + c * 4);
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(s_q + (ty * kR + i) * LD + c * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(q.x, k[j].x, fmaf(q.y, k[j].y, fmaf(q.z, k[j].z, fmaf(q.w, k[j].w, s[i][j]))));
      }
    }
    if (Sh::P_OVER_K) __syncthreads();
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = kb + tx + 16 * j;
        float x = s[i][j] * log2s;
        if (cap2 > 0.f) x = capped(x, cap2, inv_cap2);
        x -= slope2[i] * fabsf((float)(pos[i] - key));
        if (key < seen[i].lo || key >= seen[i].hi || (bad >> (tx + 16 * j) & 1)) x = -INFINITY;
        s[i][j] = x;
        mx = fmaxf(mx, x);
      }
#pragma unroll
      for (int k = 1; k <= 8; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, k));
      if (mx > m[i]) {
        const float f = ex2(m[i] - mx);
        m[i] = mx;
        l[i] *= f;
#pragma unroll
        for (int c = 0; c < OC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][c][e] *= f;
      }
      const float base = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = ex2(s[i][j] - base);
        l[i] += s[i][j];                               // this thread's keys only
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < kR; i += 4)
        *reinterpret_cast<float4*>(s_p + (tx + 16 * j) * LP + ty * kR + i) =
            make_float4(s[i][j], s[i + 1][j], s[i + 2][j], s[i + 3][j]);
    __syncwarp();                                      // a warp reads the rows it wrote
#pragma unroll 2
    for (int k = 0; k < kKeys; ++k) {
      float w[kR];
#pragma unroll
      for (int i = 0; i < kR; i += 4)
        *reinterpret_cast<float4*>(w + i) = *reinterpret_cast<const float4*>(s_p + k * LP + ty * kR + i);
#pragma unroll
      for (int c = 0; c < OC; ++c) {
        const float4 v = *reinterpret_cast<const float4*>(s_v + k * LD + c * 64 + tx * 4);
#pragma unroll
        for (int i = 0; i < kR; ++i) {
          o[i][c][0] = fmaf(w[i], v.x, o[i][c][0]);
          o[i][c][1] = fmaf(w[i], v.y, o[i][c][1]);
          o[i][c][2] = fmaf(w[i], v.z, o[i][c][2]);
          o[i][c][3] = fmaf(w[i], v.w, o[i][c][3]);
        }
      }
    }
    __syncthreads();                                   // the stage may be filled again
  }

#pragma unroll
  for (int i = 0; i < kR; ++i) {
#pragma unroll
    for (int k = 1; k <= 8; k <<= 1) l[i] += __shfl_xor_sync(FULL, l[i], k);
    const int tok = tok0 + (ty * kR + i) / G;
    if (tok >= n_r || row0 + tok >= a.n_q) continue;
    const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
    const float lse2 = l[i] > 0.f ? m[i] + lg2(l[i]) : -INFINITY;
    const size_t at = ((size_t)row0 + tok) * hq + g * G + (ty * kR + i) % G;
    const size_t part = (size_t)split * a.n_q * hq + at;
    float* dst = p.splits > 1 ? p.part_o + part * D : static_cast<float*>(a.out) + at * D;
#pragma unroll
    for (int c = 0; c < OC; ++c)
      *reinterpret_cast<float4*>(dst + c * 64 + tx * 4) =
          make_float4(o[i][c][0] * inv, o[i][c][1] * inv, o[i][c][2] * inv, o[i][c][3] * inv);
    if (tx == 0) {
      if (p.splits > 1) p.part_lse[part] = lse2;
      else if (a.lse) a.lse[at] = lse2 * LN2;
    }
  }
}

template <int D> cudaError_t launch(const PrefillArgs& p, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(prefill_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       ShapeF32<D>::SMEM);
  if (e != cudaSuccess) return e;
  prefill_f32_kernel<D><<<(unsigned)p.blocks * p.a.h_kv * p.splits, 256, ShapeF32<D>::SMEM, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess || p.splits == 1) return e;
  return launch_prefill_join<float, D>(p, s);
}

}  // namespace

cudaError_t launch_prefill_f32(const PrefillArgs& p, cudaStream_t s) {
  return p.a.head_dim == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace quest
