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
#include "append_parts.cuh"
#include "tmap.h"

namespace quest {
namespace {

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
      walk_rows<T, TG>(static_cast<const T*>(a.q) + row0 * a.q_stride + h * D, a.q_stride,
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
      walk_rows<T, TG>(static_cast<const T*>(a.k_new) + row0 * a.k_stride + h * D, a.k_stride,
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
      walk_rows<T, TG>(static_cast<const T*>(a.v_new) + row0 * a.v_stride + h * D, a.v_stride,
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
  // a CTA per SM; more of them only start more often (200 one-token requests of 8
  // KV heads: 9.5 us with 152 CTAs wanted, 13.6 with 608; 2048 tokens 11.5 and 19.3)
  const dim3 grid = append_grid(a, sms);
  if (a.dtype == QUEST_F16 && a.summary_fp8)
    return a.head_dim == 128 ? launch<__half, 128, true>(a, grid, sms, s) : launch<__half, 64, true>(a, grid, sms, s);
  if (a.dtype == QUEST_F16)
    return a.head_dim == 128 ? launch<__half, 128, false>(a, grid, sms, s) : launch<__half, 64, false>(a, grid, sms, s);
  return a.head_dim == 128 ? launch<float, 128, false>(a, grid, sms, s) : launch<float, 64, false>(a, grid, sms, s);
}

}  // namespace quest
