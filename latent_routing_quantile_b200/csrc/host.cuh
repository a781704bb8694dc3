// Host-side helpers shared by the library's sources: tensor maps and kernel launches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cstring>

#include "../../include/lmoe.h"

#define CK(x)                                 \
  do {                                        \
    if ((x) != cudaSuccess) return LMOE_ECUDA; \
  } while (0)

namespace lmoe {

constexpr int kBalMaxSeqs = 1 << 24;  // sequences of a balance loss

// ------------------------------------------------------------------ tensor maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

// Tensor map of a row-major matrix with a 128-byte swizzle (the layout the MMA descriptors and the
// staged epilogue expect).
inline bool make_map_t(CUtensorMap* m, const void* base, long long rows, long long cols, long long pitch, int box_rows,
                bool f32) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const long long es_bytes = f32 ? 4 : 2;
  if (((uintptr_t)base & 15) || ((pitch * es_bytes) & 15) || rows <= 0 || cols <= 0) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(pitch * es_bytes)};
  cuuint32_t box[2] = {f32 ? 32u : 64u, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base),
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// bf16 matrix [rows, cols], row pitch `pitch` elements; box = 64 columns (128 bytes) x box_rows.
inline bool make_map(CUtensorMap* m, const void* base, long long rows, long long cols, long long pitch, int box_rows) {
  return make_map_t(m, base, rows, cols, pitch, box_rows, false);
}
// 8-bit matrix [rows, cols]; box = 128 columns (128 bytes) x box_rows, 128-byte swizzle.
inline bool make_map_u8(CUtensorMap* m, const void* base, long long rows, long long cols, long long pitch, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  if (((uintptr_t)base & 15) || (pitch & 15) || rows <= 0 || cols <= 0) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)pitch};
  cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// fp32 matrix; box = 32 columns (128 bytes) x box_rows.
inline bool make_map_f32(CUtensorMap* m, const void* base, long long rows, long long cols, long long pitch, int box_rows) {
  return make_map_t(m, base, rows, cols, pitch, box_rows, true);
}

// Raises a kernel's dynamic shared-memory limit once per device; `done` is the caller's own
// per-kernel flag word (one bit per device).
template <typename K>
cudaError_t ensure_smem_attr(K kern, int bytes, unsigned& done) {
  int dev = 0;
  cudaGetDevice(&dev);
  const unsigned bit = 1u << (dev & 31);
  if (done & bit) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done |= bit;
  return e;
}

// The largest cluster of `kern` (blocks of `threads`, no dynamic shared memory) that the current device
// places: 16 CTAs, where it has that many SMs side by side, or 8, which every device has (a slice of a
// partitioned one may not have 16).  `known` and `large` are the caller's own per-kernel flag words (one bit
// per device): the device is asked once.
template <typename K>
int largest_cluster(K kern, int threads, std::atomic<unsigned>& known, std::atomic<unsigned>& large) {
  int dev = 0;
  cudaGetDevice(&dev);
  const unsigned bit = 1u << (dev & 31);
  if (!(known & bit)) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(threads);
    cudaLaunchAttribute attr;
    memset(&attr, 0, sizeof(attr));
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 16;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0)
      large |= bit;
    else
      cudaGetLastError();  // not the launch's
    known |= bit;
  }
  return (large & bit) ? 16 : 8;
}

// Launches `kern` with programmatic stream serialisation, so its blocks may be scheduled while
// the previous kernel of the stream drains (every kernel of the layer calls pdl_wait() before
// touching data another kernel writes), and for cluster_x > 1 in clusters of cluster_x CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_k(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, int cluster_x,
                     Args... args) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  memset(attr, 0, sizeof(attr));
  int n = 0;
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  if (cluster_x > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster_x;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// lmoe_balance_loss with S' from a device word where that is more than 0 (total: null for none), which adds
// the kernels it launched to *launches (null: not counted).
int balance_loss(const float* scores, const int32_t* idx, int32_t T, int32_t E, int32_t k, const int32_t* cu_seqlens,
                 int32_t S, const int32_t* total, float coef, int32_t* counts, float* loss, float* dscores,
                 void* scratch, uint32_t* status, void* stream, long long* launches);

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

}  // namespace lmoe
