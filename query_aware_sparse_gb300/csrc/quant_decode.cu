// Decode attention over the E4M3 cache: plan and launch (quant_decode.cuh).
#include <algorithm>
#include <atomic>

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

template <int D, int NT> cudaError_t launch_join(const DecodeArgs& p, unsigned rows, cudaStream_t s) {
  // the same shared memory split as the kernel before it
  const cudaError_t e = cudaFuncSetAttribute(dense_decode_join_kernel<D, NT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                             cudaSharedmemCarveoutMaxShared);
  return e == cudaSuccess ? launch_pdl(dense_decode_join_kernel<D, NT>, rows, NT, 0, s, p) : e;
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
  // few units have many parts: more warps take them
  const unsigned rows = (unsigned)p.a.batch * p.a.h_kv * p.a.group;
  return p.n_warps > 64 * p.a.batch * (long long)p.a.h_kv ? launch_join<D, 1024>(p, rows, s) : launch_join<D, kJoinThreads>(p, rows, s);
}

// Clusters of 1 to 8 CTAs of a kernel that the current device keeps at once
// (asked for once per device; the driver packs them into its GPCs).
template <typename K> int resident_clusters(K kernel, int ctas, size_t smem, std::atomic<int> (&known)[64][9]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 0;
  int n = known[dev][ctas].load();
  if (n) return n;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kUnitWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  known[dev][ctas].store(n > 0 ? n : -1);
  return n;
}

// CTAs of a unit's cluster: as many as the device holds at once for all units,
// with a tile for each warp. 0: the equal runs serve the call better, which cost
// 5 us more to start and join, but leave no warp with more tiles than another.
// A warp's tiles one after the other take 0.6 us each (latency) or, where the
// SMs are full, what HBM gives them. us, clusters and runs (128 dims, pages of 16):
//   1 head, 31 / 250 / 500 / 1000 pages          3.6 / 7.5 / 12.8 / 22     9.0 / 10.5 / 11.4 / 12.4
//   32 heads, 125 / 250 / 500 / 1000             7.4 / 11.3 / 18 / 33      11.9 / 16.9 / 21.8 / 31.5
//   16 requests of 8 heads, 64 / 256 / 512       10.2 / 25.2 / 45.4        16.0 / 30.5 / 50.4
// The other shapes (64 dims, pages of 32, 4 and 8 heads to a KV head) cross at the
// same number of tiles: where the rule errs it costs 16% (64 dims, 16 requests of 8
// heads, 1024 pages: 57.3 and 67.0 with 8 heads each, 58.7 and 63.6 with one), most
// often under 10%.
// More units than CTAs: the last wave is short of work and adds up to 0.6 us per
// tile (0.4 for the smallest pages); the runs cost their 5 us and 4 ns per row of q
// (a joining CTA each); over all shapes the border below errs by 14% at most. us for
// lists of pages of 16, 128 dims, 1 / 8 heads to a KV head:
//   60 requests of 8 heads, 32 pages    18.1 / 18.3    20.7 / 36.0
//     64                                32.9 / 31.5    29.0 / 44.3
//     128                               60.6 / 57.0    47.4 / 63.0
//     256                               117 / 118      84.8 / 101
//   300 requests of 8 heads, 32 pages   53.9 / 56.7    66.1 / 129
//   1000 requests of 4 heads, 16 pages  50.5 / 55.8    61.5 / 143
// Tables: the host knows no lengths, so all pages may be one request's, unless a
// window bounds what is read.
template <int D, int S, bool LIST, bool PACK> int unit_ctas(const DecodeArgs& p) {
  const long long units = (long long)p.a.batch * p.a.h_kv;
  long long most = LIST ? p.sel_k : p.a.nnz;
  if (!LIST && p.a.window > 0) most = std::min<long long>(most, (p.a.window - 1) / p.a.page_size + 2);
  static std::atomic<int> known[64][9];
  auto resident = [&](int c) {
    return resident_clusters(quant_unit_kernel<D, S, LIST, PACK>, c, UnitShape<D, S>::SMEM, known);
  };
  int c = 8;
  while (c > 1 && (most < kUnitWarps * c || units > resident(c))) --c;
  const int n = resident(c), sms = sm_count();
  if (n <= 0) return 0;
  const long long waves = (units + n - 1) / n, tiles = (most + kUnitWarps * c - 1) / (kUnitWarps * c);
  if (waves > 1) return tiles <= 12 + units * p.a.group / 150 ? c : 0;
  return tiles <= (units * c >= 2 * sms ? 64 : units * c >= sms ? 20 : 12) ? c : 0;
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

template <int D, int S, bool LIST, bool PACK> cudaError_t launch_either(const DecodeArgs& p, cudaStream_t s) {
  const int ctas = unit_ctas<D, S, LIST, PACK>(p);
  return ctas ? launch_units<D, S, LIST, PACK>(p, ctas, s) : launch<D, S, LIST, PACK>(p, s);
}

template <bool LIST, bool PACK> cudaError_t launch_shape(const DecodeArgs& p, cudaStream_t s) {
  if (p.a.head_dim == 128)
    return p.a.page_size == 16 ? launch_either<128, 16, LIST, PACK>(p, s) : launch_either<128, 32, LIST, PACK>(p, s);
  return p.a.page_size == 16 ? launch_either<64, 16, LIST, PACK>(p, s) : launch_either<64, 32, LIST, PACK>(p, s);
}
template <bool LIST> cudaError_t launch_group(const DecodeArgs& p, cudaStream_t s) {
  return p.a.group <= 4 ? launch_shape<LIST, true>(p, s) : launch_shape<LIST, false>(p, s);
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
  return sel_logical ? launch_group<true>(p, s) : launch_group<false>(p, s);
}

}  // namespace quest
