// Decode attention over the E4M3 cache: plan and launch (quant_decode.cuh).
#include <algorithm>

#include "quant_decode.cuh"
#include "internal.h"
#include "tmap.h"

namespace quest {
namespace {

struct Plan { int warps; size_t part_o, part_ml, bytes; };

Plan plan_quant(int32_t batch, int32_t h_kv, int32_t group, int32_t head_dim) {
  Plan p;
  p.warps = sm_count() * (head_dim == 64 ? RecordShape<64, 16>::WARPS : RecordShape<128, 16>::WARPS);
  const size_t slots = ((size_t)p.warps + (size_t)batch * h_kv) * group;
  p.part_o = (((size_t)batch + 1) * sizeof(long long) + 255) & ~(size_t)255;
  p.part_ml = p.part_o + slots * head_dim * sizeof(float);
  p.bytes = p.part_ml + slots * sizeof(float2);
  return p;
}

template <int D, int S, bool LIST, bool PACK>
cudaError_t launch(const DecodeArgs& p, cudaStream_t s) {
  using W = WarpE4M3<D, S, PACK>;
  using Sh = typename W::Shape;
  static_assert(Sh::WARPS == RecordShape<D, 16>::WARPS, "one plan for both page sizes");
  cudaError_t e = cudaFuncSetAttribute(dense_decode_kernel<W, D, LIST>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
  if (e != cudaSuccess) return e;
  const PageRecords src{static_cast<const uint8_t*>(p.a.k_pool)};
  e = launch_pdl(dense_decode_kernel<W, D, LIST>, p.n_warps / Sh::WARPS, Sh::WARPS * 32, Sh::SMEM, s, src, p);
  if (e != cudaSuccess) return e;
  // the same shared memory split as the kernel before it
  e = cudaFuncSetAttribute(dense_decode_join_kernel<D>, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  return launch_pdl(dense_decode_join_kernel<D>, (unsigned)p.a.batch * p.a.h_kv * p.a.group, kJoinThreads, 0, s, p);
}

// CTAs of a unit's cluster: as many as the device holds at once for all units,
// with a tile for each warp. 0: the equal runs serve the call better, which cost
// 5 us more to start and join, but leave no warp with more tiles than another.
// A warp's tiles one after the other take 0.6 us each (latency) or, from a CTA
// per SM on, what HBM gives them. us, clusters and runs (128 dims, pages of 16):
//   1 head, 31 / 250 / 500 / 1000 pages   3.8 / 7.9 / 12.8 / 22   9.0 / 10.7 / 11.5 / 12.6
//   32 heads, 125 / 250 / 500 / 1000      7.6 / 11.6 / 18.6 / 33  11.9 / 16.9 / 21.9 / 31.7
//   16 requests of 8 heads, 32 / 128 / 256 / 512 listed   7.8 / 18.5 / 32 / 61   11.8 / 21.3 / 30 / 50
//   64 of 8, 8 / 32 / 128 (two waves)     8.0 / 19.6 / 63         12.2 / 21.1 / 50
// Tables: the host knows no lengths, so all pages may be one request's, unless a
// window bounds what is read.
template <bool LIST> int unit_ctas(const DecodeArgs& p) {
  const long long units = (long long)p.a.batch * p.a.h_kv;
  long long most = LIST ? p.sel_k : p.a.nnz;
  if (!LIST && p.a.window > 0) most = std::min<long long>(most, (p.a.window - 1) / p.a.page_size + 2);
  const int sms = sm_count(), slots = kUnitCtasPerSm * sms;
  int c = 8;
  while (c > 1 && (units * c > slots || most < kUnitWarps * c)) c /= 2;
  const long long waves = (units * c + slots - 1) / slots, tiles = (most + kUnitWarps * c - 1) / (kUnitWarps * c);
  return waves * tiles <= (units * c >= sms ? 20 : 12) ? c : 0;
}

template <int D, int S, bool LIST, bool PACK>
cudaError_t launch_units(const DecodeArgs& p, int ctas, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(quant_unit_kernel<D, S, LIST, PACK>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, UnitShape<D, S>::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl_clusters(quant_unit_kernel<D, S, LIST, PACK>, (unsigned)p.a.batch * p.a.h_kv * ctas, ctas,
                             kUnitWarps * 32, UnitShape<D, S>::SMEM, s,
                             PageRecords{static_cast<const uint8_t*>(p.a.k_pool)}, p);
}

template <int D, int S, bool LIST> cudaError_t launch_either(const DecodeArgs& p, cudaStream_t s) {
  const int ctas = unit_ctas<LIST>(p);
  if constexpr (S == 32)
    if (p.a.group <= 4) return ctas ? launch_units<D, S, LIST, true>(p, ctas, s) : launch<D, S, LIST, true>(p, s);
  return ctas ? launch_units<D, S, LIST, false>(p, ctas, s) : launch<D, S, LIST, false>(p, s);
}

template <bool LIST> cudaError_t launch_shape(const DecodeArgs& p, cudaStream_t s) {
  if (p.a.head_dim == 128)
    return p.a.page_size == 16 ? launch_either<128, 16, LIST>(p, s) : launch_either<128, 32, LIST>(p, s);
  return p.a.page_size == 16 ? launch_either<64, 16, LIST>(p, s) : launch_either<64, 32, LIST>(p, s);
}

}  // namespace

size_t quant_decode_workspace(int32_t batch, int32_t h_kv, int32_t group, int32_t head_dim) {
  return plan_quant(batch, h_kv, group, head_dim).bytes;
}

cudaError_t launch_quant_decode(const DenseArgs& a, const int32_t* sel_logical, const int32_t* sel_phys,
                                int32_t k, cudaStream_t s) {
  const Plan plan = plan_quant(a.batch, a.h_kv, a.group, a.head_dim);
  char* ws = static_cast<char*>(a.workspace);
  DecodeArgs p{};
  p.a = a;
  p.sel_logical = sel_logical;
  p.sel_phys = sel_phys;
  p.sel_k = k;
  p.min_run = 4;
  p.starts = reinterpret_cast<long long*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + plan.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + plan.part_ml);
  p.n_warps = plan.warps;
  p.wait_limit = wait_limit();
  return sel_logical ? launch_shape<true>(p, s) : launch_shape<false>(p, s);
}

}  // namespace quest
