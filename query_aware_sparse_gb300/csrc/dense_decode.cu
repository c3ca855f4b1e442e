// Dense decode attention: plan, tensor maps and launch (dense_decode.cuh).
#include "dense_decode.cuh"
#include "internal.h"
#include "tmap.h"

namespace quest {
namespace {

struct Plan { int warps; size_t part_o, part_ml, bytes; };

Plan plan_decode(int32_t batch, int32_t h_kv, int32_t group, int32_t head_dim, int32_t dtype) {
  Plan p;
  p.warps = sm_count() * (dtype != QUEST_F16 ? DecodeShape<float, 64>::WARPS
                          : head_dim == 64   ? DecodeShape<__half, 64>::WARPS
                                             : DecodeShape<__half, 128>::WARPS);
  const size_t slots = ((size_t)p.warps + (size_t)batch * h_kv) * group;
  p.part_o = (((size_t)batch + 1) * sizeof(long long) + 255) & ~(size_t)255;
  p.part_ml = p.part_o + slots * head_dim * sizeof(float);
  p.bytes = p.part_ml + slots * sizeof(float2);
  return p;
}

static_assert(DecodeShape<float, 64>::WARPS == DecodeShape<float, 128>::WARPS, "one plan for fp32");

template <typename W, int D>
cudaError_t launch(const DecodeMaps& maps, const DecodeArgs& p, cudaStream_t s) {
  using Sh = typename W::Shape;
  cudaError_t e = cudaFuncSetAttribute(dense_decode_kernel<W, D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(dense_decode_kernel<W, D>, p.n_warps / Sh::WARPS, Sh::WARPS * 32, Sh::SMEM, s, maps, p);
  if (e != cudaSuccess) return e;
  // the same shared memory split as the kernel before it
  e = cudaFuncSetAttribute(dense_decode_join_kernel<D>, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  return launch_pdl(dense_decode_join_kernel<D>, (unsigned)p.a.batch * p.a.h_kv * p.a.group, kJoinThreads, 0, s, p);
}

template <int D> cudaError_t launch_f32(const DecodeMaps& maps, const DecodeArgs& p, cudaStream_t s) {
  switch (p.a.group) {
    case 1: return launch<WarpF32<D, 1>, D>(maps, p, s);
    case 2: return launch<WarpF32<D, 2>, D>(maps, p, s);
    case 4: return launch<WarpF32<D, 4>, D>(maps, p, s);
    default: return launch<WarpF32<D, 8>, D>(maps, p, s);
  }
}

}  // namespace

size_t dense_decode_workspace(int32_t batch, int32_t, int32_t h_kv, int32_t group,
                              int32_t head_dim, int32_t, int32_t dtype) {
  return plan_decode(batch, h_kv, group, head_dim, dtype).bytes;
}

cudaError_t launch_dense_decode(const DenseArgs& a, cudaStream_t s) {
  const Plan plan = plan_decode(a.batch, a.h_kv, a.group, a.head_dim, a.dtype);
  char* ws = static_cast<char*>(a.workspace);
  DecodeArgs p{};
  p.a = a;
  p.starts = reinterpret_cast<long long*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + plan.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + plan.part_ml);
  p.n_warps = plan.warps;
  p.min_run = 4;
  p.wait_limit = wait_limit();
  DecodeMaps maps;
  const int rows = a.dtype == QUEST_F16 ? 16 : 8;
  if (!encode_pool(&maps.k, a, a.k_pool, rows) || !encode_pool(&maps.v, a, a.v_pool, rows))
    return cudaErrorInvalidValue;
  if (a.dtype == QUEST_F16)
    return a.head_dim == 128 ? launch<WarpF16<128>, 128>(maps, p, s) : launch<WarpF16<64>, 64>(maps, p, s);
  return a.head_dim == 128 ? launch_f32<128>(maps, p, s) : launch_f32<64>(maps, p, s);
}

}  // namespace quest
