// Normed and E4M3 appends: launch (norm_append.cuh, one file per store and head dim).
#include "append_parts.cuh"
#include "quant.h"
#include "tmap.h"

namespace quest {

cudaError_t launch_norm_append(const NormAppendArgs& args, bool e4m3, cudaStream_t s) {
  NormAppendArgs p = args;
  const int sms = sm_count();
  // A CTA per SM, as in rope_append.cu; with more work than that (over 6 steps
  // of 4 KB for each of the 16 warps that an SM holds) five, so that the last ones
  // are short. us with one and with five, fp16 and into E4M3, by steps per warp:
  //   22 requests of 150 tokens, 32 heads of 8, 64 dims   14    66 -> 60, 69 -> 63
  //   8192 tokens, 8 heads of 4                           10    42.5 -> 38.5, 44.0 -> 40.9
  //   2600 tokens, 40 heads                                8    45 -> 35, 48 -> 39
  //   4096 tokens, 8 heads of 4                            5    21.9 -> 21.8, 22.8 -> 22.3
  //   2048 tokens, 8 heads of 4                            2.5  12.2 -> 13.9, 12.9 -> 15.5
  // and 14400 fp32 tokens, 8 heads of 2 (24): 89 -> 81.
  const long long row = (long long)p.a.head_dim * (p.a.dtype == QUEST_F16 ? 2 : 4);
  const long long rows = (long long)p.a.h_kv * ((p.a.q ? p.a.group : 0) + 2) * p.a.n_new;
  const dim3 grid = append_grid(p.a, rows * row / 4096 > 6LL * 16 * sms ? 5LL * sms : sms);
  const bool d128 = p.a.head_dim == 128;
  if (e4m3) return d128 ? launch_norm_append_e4m3_d128(p, grid, sms, s) : launch_norm_append_e4m3_d64(p, grid, sms, s);
  if (p.a.dtype == QUEST_F32) return launch_norm_append_f32(p, grid, sms, s);
  return d128 ? launch_norm_append_f16_d128(p, grid, sms, s) : launch_norm_append_f16_d64(p, grid, sms, s);
}

}  // namespace quest
