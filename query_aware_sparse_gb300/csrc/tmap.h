// Tensor maps of the paged pools for tiled TMA loads (host side).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdlib.h>

#include "dense.h"

namespace quest {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled tensor_map_encoder() {
  static const EncodeTiled f = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<EncodeTiled>(fn);
  }();
  return f;
}

// A map with dense strides of 16-byte rows, boxes of 128-byte rows, 128-byte swizzle.
inline bool encode_map(CUtensorMap* m, int32_t dtype, const void* base, int rank,
                       const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t one[3] = {1, 1, 1};
  const EncodeTiled f = tensor_map_encoder();
  return f && f(m, dtype == QUEST_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                rank, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// K or V pool as rows of one token and KV head: boxes of `rows` rows, 128 bytes each.
inline bool encode_pool(CUtensorMap* m, const DenseArgs& a, const void* pool, int rows) {
  const cuuint64_t size = a.dtype == QUEST_F16 ? 2 : 4;
  const cuuint64_t dims[2] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.n_phys * a.h_kv * a.page_size};
  const cuuint64_t strides[1] = {(cuuint64_t)a.head_dim * size};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)rows};
  return encode_map(m, a.dtype, pool, 2, dims, strides, box);
}

inline int sm_count() {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaGetLastError();
  return sms;
}

// A launch that may begin before the kernel in front of it on the stream has
// ended (it waits with pdl_wait), in clusters of `ctas` CTAs where that is not 0.
template <typename K, typename... A>
inline cudaError_t launch_pdl_clusters(K kernel, unsigned grid, unsigned ctas, unsigned threads, size_t smem,
                                       cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  static const bool off = getenv("QUEST_NO_PDL") != nullptr;
  if (!off) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (ctas) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = ctas;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename K, typename... A>
inline cudaError_t launch_pdl(K kernel, unsigned grid, unsigned threads, size_t smem, cudaStream_t s, A... args) {
  return launch_pdl_clusters(kernel, grid, 0, threads, smem, s, args...);
}

}  // namespace quest
