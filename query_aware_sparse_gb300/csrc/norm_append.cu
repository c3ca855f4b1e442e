// Normed and E4M3 appends: launch (norm_append.cuh, one file per store).
#include "append_parts.cuh"
#include "quant.h"
#include "tmap.h"

namespace quest {

cudaError_t launch_norm_append(const NormAppendArgs& args, bool e4m3, cudaStream_t s) {
  NormAppendArgs p = args;
  const int sms = sm_count();
  const dim3 grid = append_grid(p.a, sms);
  if (e4m3) return launch_norm_append_e4m3(p, grid, sms, s);
  return p.a.dtype == QUEST_F16 ? launch_norm_append_f16(p, grid, sms, s) : launch_norm_append_f32(p, grid, sms, s);
}

}  // namespace quest
