// The E4M3 cache read back into fp16 pages of another pool.
//
// Every stored value, code * 2^e, is an fp16 number: nothing is rounded. Bound:
// HBM, 2 (D + 1) bytes read and 4 D written a token and KV head.
//
// Split. A warp takes one page of one KV head: 16 bytes per lane and load, as
// the record lays them out (e4m3_page.cuh), K's as 32 bytes of one token, V's as
// 8 bytes of four tokens, which eight lanes make 64 bytes of a row.
//
// Measured: 65536 tokens of 8 heads (128 dims) 68 us, 5920 GB/s (88% of the rate of
// a copy, which writes as much as it reads; here two thirds are writes). V in 16
// bytes of two tokens, traded between lanes: 71 us; CTAs of four warps: 68.
#include "e4m3_page.cuh"
#include "dense.cuh"
#include "quant.h"

namespace quest {
namespace {

constexpr int kReadWarps = 8;

// The request that owns table entry e: the last one that starts at or before
// it, 32 at a time.
__device__ __forceinline__ int request_of_entry(const int32_t* page_indptr, int batch, int e, int lane) {
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const int c = __popc(__ballot_sync(FULL, lane * step < n && page_indptr[i] <= e)) - 1;
    lo += max(c, 0) * step;
    n = min(step, batch - lo);
  }
  return lo;
}

template <int D, int S>
__global__ void __launch_bounds__(kReadWarps * 32) quant_read_kernel(const QuantReadArgs a) {
  constexpr size_t REC = record_bytes(S, D);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0)                                 // tokens that no entry holds
    for (int r = threadIdx.x; r < a.batch; r += kReadWarps * 32)
      held_tokens(a.seq_lens[r], a.page_indptr[r + 1] - a.page_indptr[r], S, a.err);
  const long long item = (long long)blockIdx.x * kReadWarps + warp;
  const int e = (int)(item / a.h_kv), head = (int)(item % a.h_kv);
  if (e >= a.nnz) return;
  const int r = request_of_entry(a.page_indptr, a.batch, e, lane);
  const int lp = e - a.page_indptr[r];
  if (lp < 0 || e >= a.page_indptr[r + 1]) return;     // an entry of no request
  const int n = min(S, max(0, a.seq_lens[r]) - min(lp, 0x7fffffff / S) * S);
  if (n <= 0) return;
  const int src = a.page_indices[e], dst = a.dst_indices ? a.dst_indices[e] : e;
  if (src < 0 || src >= a.n_phys || dst < 0 || dst >= a.n_dst) {
    if (lane == 0) report(a.err, QUEST_DEVERR_PAGE_RANGE);
    return;
  }
  const uint8_t* rec = a.pool + ((size_t)src * a.h_kv + head) * REC;
  const size_t row = ((size_t)dst * a.h_kv + head) * S * D;
  __half* k = static_cast<__half*>(a.k_out) + row;
  __half* v = static_cast<__half*>(a.v_out) + row;
  const int g = lane >> 2, t = lane & 3;
  constexpr int KC = S * D / 512, VC = S * D / 512;
  uint4 x[KC], y[VC];
#pragma unroll
  for (int i = 0; i < KC; ++i) x[i] = ld_stream_v4(rec + i * 512 + lane * 16);
#pragma unroll
  for (int i = 0; i < VC; ++i) y[i] = ld_stream_v4(rec + S * D + i * 512 + lane * 16);
  const uint8_t* scales = rec + 2 * S * D;
#pragma unroll
  for (int i = 0; i < KC; ++i) {                       // eight tokens of 64 dims
    const int tok = i * 8 % S + g, dim = i * 8 / S * 64 + 16 * t;
    const uint32_t f = scale_h2(scales[tok] * 0x00010001u);
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t o[8];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      o[2 * c] = mul_h2(e4m3_pair(w[c]), f);
      o[2 * c + 1] = mul_h2(e4m3_pair(w[c] >> 16), f);
    }
    if (tok < n) {
      st_v4(k + tok * D + dim, make_uint4(o[0], o[1], o[2], o[3]));
      st_v4(k + tok * D + dim + 8, make_uint4(o[4], o[5], o[6], o[7]));
    }
  }
#pragma unroll
  for (int s = 0; s < S / 16; ++s) {
    const int tok = 16 * s + 2 * t;
    const uint32_t f0 = scale_h2(scales[S + tok] | (uint32_t)scales[S + tok + 1] << 16);
    const uint32_t f1 = scale_h2(scales[S + tok + 8] | (uint32_t)scales[S + tok + 9] << 16);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {                 // 16 tokens of 32 dims
      const uint4 c = y[s * (D / 32) + i];
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
      uint32_t p[4], q[4];                             // a dim's values of tokens 2 t, + 1; + 8, + 9
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        p[d] = mul_h2(e4m3_pair(w[d]), f0);
        q[d] = mul_h2(e4m3_pair(w[d] >> 16), f1);
      }
      __half* at = v + tok * D + 32 * i + 4 * g;
      if (tok < n) st_v2(at, make_uint2(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410)));
      if (tok + 1 < n) st_v2(at + D, make_uint2(__byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632)));
      if (tok + 8 < n) st_v2(at + 8 * D, make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410)));
      if (tok + 9 < n) st_v2(at + 9 * D, make_uint2(__byte_perm(q[0], q[1], 0x7632), __byte_perm(q[2], q[3], 0x7632)));
    }
  }
}

}  // namespace

cudaError_t launch_quant_read(const QuantReadArgs& a, cudaStream_t s) {
  const long long items = (long long)a.nnz * a.h_kv;
  const unsigned grid = (unsigned)((items + kReadWarps - 1) / kReadWarps);
  const bool d128 = a.head_dim == 128, s16 = a.page_size == 16;
  auto kernel = d128 ? (s16 ? quant_read_kernel<128, 16> : quant_read_kernel<128, 32>)
                     : (s16 ? quant_read_kernel<64, 16> : quant_read_kernel<64, 32>);
  kernel<<<grid > 0 ? grid : 1, kReadWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace quest
