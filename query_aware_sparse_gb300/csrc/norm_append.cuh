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
// bytes are stored by themselves (a code's byte belongs to one token). HBM bound
// for prompts, latency bound for decode steps.
#pragma once

#include "append_parts.cuh"
#include "e4m3_page.cuh"
#include "quant.h"
#include "tmap.h"

namespace quest {

template <typename T, int D, bool E4, bool F8, bool IL, int NT>
__global__ void __launch_bounds__(NT, 512 / NT) norm_append_kernel(const NormAppendArgs p) {
  static_assert(sizeof(T) == 2 || !(E4 || F8), "8-bit codes are made of fp16 rows");
  constexpr int VEC = Elem<T>::kVec;
  constexpr int PC = D / VEC / 2;               // lanes per token: pairs of 16-byte pieces
  constexpr int TG = 32 / PC;                   // tokens side by side
  constexpr int U = 4;                          // of which so many are in flight
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

  if (half > 0) {
    const int jj = threadIdx.x % half;
    const unsigned long long f = turn_fraction(a.inv_freq[jj]);
    for (int t = threadIdx.x / half; t < ntok && threadIdx.x < NT / half * half; t += NT / half) {
      const int pos = a.positions ? a.positions[row0 + t] : t_begin + t;
      const int turn = (int)(((unsigned long long)(long long)pos * f) >> 32);   // half turns in 2^-31
      float sn, cs;
      sincospif((float)turn * 0x1p-31f, &sn, &cs);
      s_cos[t * (D / 2) + jj] = cs;
      s_sin[t * (D / 2) + jj] = sn;
    }
  }
  const int pp = page_of(a, r, lp);
  __syncthreads();

  const int h0 = blockIdx.y * a.heads_per_cta, h1 = min(a.h_kv, h0 + a.heads_per_cta);
  const int nh = h1 - h0;
  const int qn = a.q ? nh * a.group : 0;        // rows: queries, then keys, then values
  const int slot0 = t_begin - lp * S;
  const bool fresh = slot0 == 0;
  const size_t page = (size_t)max(pp, 0) * a.h_kv;
  const size_t rec = record_bytes(S, D);
  constexpr size_t SE = F8 ? 1 : sizeof(T);     // bytes of a summary element
  bool ovf = false;

  const int lane = threadIdx.x & 31, it = threadIdx.x % PC, tg = lane / PC;
  int ca = 2 * it, cb = 2 * it + 1;             // the lane's pieces, and whether they turn
  bool turn = ca * VEC < a.rotary_dim;
  if (!IL) {
    turn = it * VEC < half;
    if (turn) { ca = it; cb = it + half / VEC; }
  }
  ca *= VEC;
  cb *= VEC;

  // Tokens t0 + u TG + tg of one head, normed (with a weight) and turned; `each`
  // gets them as stored, on all lanes of a token or none.
  auto heads = [&](const T* src, int64_t stride, const float* weight, auto each) {
    float w[2 * VEC];
    if (weight) {
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        *reinterpret_cast<float4*>(w + e) = *reinterpret_cast<const float4*>(weight + ca + e);
        *reinterpret_cast<float4*>(w + VEC + e) = *reinterpret_cast<const float4*>(weight + cb + e);
      }
    }
    for (int t0 = 0; t0 < ntok; t0 += U * TG) {
      uint4 x[U], y[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * TG + tg;
        x[u] = y[u] = make_uint4(0u, 0u, 0u, 0u);
        if (t < ntok) {
          x[u] = ld_v4(src + t * stride + ca);
          y[u] = ld_v4(src + t * stride + cb);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t0 + u * TG >= ntok) break;         // the whole warp
        const int t = t0 + u * TG + tg;
        if (weight || turn) {
          float v[2 * VEC];
          unpack16<T>(x[u], v);
          unpack16<T>(y[u], v + VEC);
          if (weight) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) ss = fmaf(v[e], v[e], ss);
            // of one token's lanes: all of them are here (the weight is the warp's)
#pragma unroll
            for (int o = 1; o < PC; o <<= 1) ss += __shfl_xor_sync(FULL, ss, o);
            const float f = rsqrtf(fmaf(ss, 1.f / D, p.eps));
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) v[e] *= f * w[e];
          }
          if (turn) {
            const int at = min(t, ntok - 1) * (D / 2) + it * VEC;
            turn_pairs<T, IL>(v, s_cos + at, s_sin + at);
          }
          x[u] = Pack<T>::pack(v);
          y[u] = Pack<T>::pack(v + VEC);
        }
        __syncwarp();
        each(x[u], y[u], t, t < ntok);
      }
    }
  };

  constexpr int VS = E4 ? 16 : kMaxPage;        // tokens of a row of values
  const int v_rows = E4 ? S / VS : 1;
  for (int row = threadIdx.x / 32; row < qn + (1 + v_rows) * nh; row += NT / 32) {
    if (row < qn) {
      const int h = h0 * a.group + row;
      const int64_t out_stride = (int64_t)a.h_kv * a.group * D;
      T* out = static_cast<T*>(a.q_out) + row0 * out_stride + h * D;
      const float* w = p.q_weight ? p.q_weight + (p.q_per_head ? h * D : 0) : nullptr;
      heads(static_cast<const T*>(a.q) + row0 * a.q_stride + h * D, a.q_stride, w,
            [&](uint4 x, uint4 y, int t, bool there) {
              if (there) {
                st_v4(out + t * out_stride + ca, x);
                st_v4(out + t * out_stride + cb, y);
              }
            });
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
      const float* w = p.k_weight ? p.k_weight + (p.k_per_head ? h * D : 0) : nullptr;
      const T* src = static_cast<const T*>(a.k_new) + row0 * a.k_stride + h * D;
      if constexpr (E4) {
        uint8_t* to = static_cast<uint8_t*>(a.k_pool) + (page + h) * rec;
        heads(src, a.k_stride, w, [&](uint4 x, uint4 y, int t, bool there) {
          uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
          auto largest = [&] {
            uint32_t m = 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max_magnitude(m, v[e]);
            m = max(m & 0xffffu, m >> 16);
#pragma unroll
            for (int o = 1; o < PC; o <<= 1) m = max(m, __shfl_xor_sync(FULL, m, o));
            return m;
          };
          uint32_t top = largest();
          if (__any_sync(FULL, top > kScaleTop)) {
            ovf = ovf || top > kScaleTop;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = keepable(v[e]);
            top = largest();
          }
          const int ex = scale_exponent(top);
          const uint32_t down = pow2_h2(-ex), up = pow2_h2(ex);
          uint32_t c[4], s[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t lo = e4m3_codes(mul_h2(v[2 * e], down)), hi = e4m3_codes(mul_h2(v[2 * e + 1], down));
            c[e] = lo | hi << 16;
            s[2 * e] = mul_h2(e4m3_pair(lo), up);
            s[2 * e + 1] = mul_h2(e4m3_pair(hi), up);
          }
          if (there) {
            const int slot = slot0 + t;
            st_v2(to + k_code_at(S, slot, ca), make_uint2(c[0], c[1]));
            st_v2(to + k_code_at(S, slot, cb), make_uint2(c[2], c[3]));
            if (it == 0) to[2 * S * D + slot] = (uint8_t)(127 + ex);
            ba.fold(make_uint4(s[0], s[1], s[2], s[3]));
            bb.fold(make_uint4(s[4], s[5], s[6], s[7]));
          }
        });
      } else {
        T* to = static_cast<T*>(a.k_pool) + ((page + h) * S + slot0) * D;
        heads(src, a.k_stride, w, [&](uint4 x, uint4 y, int t, bool there) {
          if (there) {
            st_v4(to + t * D + ca, x);
            st_v4(to + t * D + cb, y);
            ba.fold(x);
            bb.fold(y);
          }
        });
      }
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
    } else if constexpr (E4) {
      const int i0 = row - qn - nh, h = h0 + i0 / v_rows, sub = i0 % v_rows;
      if (slot0 + ntok <= sub * 16 || slot0 >= sub * 16 + 16) continue;
      const int g = lane >> 2, t = lane & 3;
      const T* src = static_cast<const T*>(a.v_new) + row0 * a.v_stride + h * D + 4 * g;
      uint8_t* to = static_cast<uint8_t*>(a.k_pool) + (page + h) * rec + S * D;
      uint2 x[4][D / 32];
      bool there[4];
      uint32_t top2[2];                         // of tokens 0, 1 and of 2, 3
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int tok = sub * 16 + (k >> 1) * 8 + 2 * t + (k & 1) - slot0;
        there[k] = tok >= 0 && tok < ntok;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          x[k][i] = make_uint2(0u, 0u);
          if (there[k]) x[k][i] = *reinterpret_cast<const uint2*>(src + tok * a.v_stride + 32 * i);
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
      const uint32_t over = __vcmpgtu2(__vmaxu2(top2[0], top2[1]), kScaleTop * 0x00010001u);
      if (__any_sync(FULL, over != 0u)) {
        ovf = ovf || over != 0u;
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
        uint32_t c[4];                          // a token's codes of four dims
#pragma unroll
        for (int k = 0; k < 4; ++k)
          c[k] = e4m3_codes(mul_h2(x[k][i].x, down[k])) | e4m3_codes(mul_h2(x[k][i].y, down[k])) << 16;
        uint8_t* at = to + ((sub * (D / 32) + i) * 32 + lane) * 16;
        if (all) {                              // a dim's codes of four tokens
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
          if (there[k]) to[S * D + S + sub * 16 + (k >> 1) * 8 + 2 * t + (k & 1)] = (uint8_t)(127 + ex[k]);
      }
    } else {
      const int h = h0 + row - qn - nh;
      walk_rows<T, TG>(static_cast<const T*>(a.v_new) + row0 * a.v_stride + h * D, a.v_stride,
                       static_cast<T*>(a.v_pool) + ((page + h) * S + slot0) * D, D, ca, cb, tg, ntok,
                       [](uint4&, uint4&, int) {});
    }
  }
  if ((E4 || F8) && ovf) report(a.err, QUEST_DEVERR_FP8_RANGE);
}

template <typename T, int D, bool E4, bool F8, int NT>
cudaError_t launch_norm_append_n(const NormAppendArgs& p, dim3 grid, cudaStream_t s) {
  if (p.a.interleaved) norm_append_kernel<T, D, E4, F8, true, NT><<<grid, NT, 0, s>>>(p);
  else norm_append_kernel<T, D, E4, F8, false, NT><<<grid, NT, 0, s>>>(p);
  return cudaGetLastError();
}
// Four warps per CTA for many CTAs of few rows, as in rope_append.cu.
template <typename T, int D, bool E4, bool F8>
cudaError_t launch_norm_append_t(const NormAppendArgs& p, dim3 grid, int sms, cudaStream_t s) {
  const int rows = p.a.heads_per_cta * ((p.a.q ? p.a.group : 0) + 2);
  const bool small = rows <= 16 && (long long)grid.x * grid.y > 4LL * sms;
  return small ? launch_norm_append_n<T, D, E4, F8, 128>(p, grid, s)
               : launch_norm_append_n<T, D, E4, F8, 256>(p, grid, s);
}

}  // namespace quest
