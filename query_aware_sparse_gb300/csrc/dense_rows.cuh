// Attention of query rows over the page table, one CTA per (row, query head):
// tiles of 128 keys, one key's logit per thread, an online softmax over the
// tiles, then one output dim per thread.
#pragma once

#include "dense.cuh"

namespace quest {

constexpr int kRowThreads = 128;

template <typename T, typename O, int D>
__global__ void __launch_bounds__(kRowThreads) dense_rows_kernel(const DenseArgs a) {
  constexpr int VEC = Elem<T>::kVec;
  __shared__ float s_q[D], s_p[kRowThreads], s_red[4];
  __shared__ const T* s_v[kRowThreads];
  const int row = blockIdx.x, h = blockIdx.y, g = h / a.group, hq = a.h_kv * a.group;
  int r = row, n = 1, i = 0;
  if (a.q_indptr) {
    for (r = 0; r < a.batch && row >= a.q_indptr[r + 1]; ++r) {}
    if (r == a.batch) return;
    n = a.q_indptr[r + 1] - a.q_indptr[r];
    i = row - a.q_indptr[r];
  }
  const int e0 = a.page_indptr[r];
  const int full = a.seq_lens[r];
  const int len = held_tokens(full, a.page_indptr[r + 1] - e0, a.page_size, a.err);
  const int pos = full - n + i;
  const Seen seen = seen_keys(pos, len, a.window, a.doc_starts ? a.doc_starts[row] : 0,
                              a.prefix_lens ? a.prefix_lens[r] : 0);
  const float slope = a.slopes ? a.slopes[h] : 0.f;
  for (int d = threadIdx.x; d < D; d += kRowThreads)
    s_q[d] = Elem<T>::to_f(static_cast<const T*>(a.q)[((size_t)row * hq + h) * D + d]);
  __syncthreads();
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int j0 = seen.lo; j0 < seen.hi; j0 += kRowThreads) {
    const int j = j0 + threadIdx.x;
    float x = -INFINITY;
    s_v[threadIdx.x] = nullptr;
    if (j < seen.hi) {
      const int pp = a.page_indices[e0 + j / a.page_size];
      if (pp < 0 || pp >= a.n_phys) {
        report(a.err, QUEST_DEVERR_PAGE_RANGE);
      } else {
        const size_t at = (((size_t)pp * a.h_kv + g) * a.page_size + j % a.page_size) * D;
        const T* k = static_cast<const T*>(a.k_pool) + at;
        s_v[threadIdx.x] = static_cast<const T*>(a.v_pool) + at;
        float s = 0.f;
        for (int c = 0; c < D; c += VEC) {
          float f[VEC];
          unpack16<T>(ld_nc_v4(k + c), f);
#pragma unroll
          for (int e = 0; e < VEC; ++e) s = fmaf(f[e], s_q[c + e], s);
        }
        x = s * a.scale;
        if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
        x -= slope * fabsf((float)(pos - j));
      }
    }
    float mx = warp_max(x);
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float mn = fmaxf(m, mx);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float p = expf(x - base), alpha = expf(m - base);
    s_p[threadIdx.x] = p;
    const float sum = warp_sum(p);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = sum;
    __syncthreads();
    l = l * alpha + s_red[0] + s_red[1] + s_red[2] + s_red[3];
    m = mn;
    o *= alpha;
    if (threadIdx.x < D) {
      const int cnt = min(kRowThreads, seen.hi - j0);
      for (int t = 0; t < cnt; ++t)
        if (s_v[t]) o = fmaf(s_p[t], Elem<T>::to_f(s_v[t][threadIdx.x]), o);
    }
    __syncthreads();
  }
  const size_t at = (size_t)row * hq + h;
  if (threadIdx.x < D)
    static_cast<O*>(a.out)[at * D + threadIdx.x] = (O)(l > 0.f ? o / l : 0.f);
  if (threadIdx.x == 0 && a.lse) a.lse[at] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace quest
