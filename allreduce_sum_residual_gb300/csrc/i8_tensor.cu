// The tensor-core products' tensor maps and launches (i8_tensor.cuh).
#include <mutex>

#include "i8_tensor.cuh"

namespace arn {

static I8Tensor i8_tensor(int type, int tokens, bool pair, bool gated) {
  return type == AR_TYPE_F32    ? i8_tensor_f32(tokens, pair, gated)
         : type == AR_TYPE_BF16 ? i8_tensor_bf16(tokens, pair, gated)
                                : i8_tensor_f16(tokens, pair, gated);
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled g_encode = nullptr;

int ready_i8_tensor(int sms, const int **pairs) {
  static std::mutex mu;
  static int of_device[kMaxDevices][3];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return AR_ERR_CUDA;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (of_device[dev][0] == 0) {
    if (g_encode == nullptr) {
      void *fn = nullptr;
      cudaDriverEntryPointQueryResult found;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                           &found) != cudaSuccess ||
          found != cudaDriverEntryPointSuccess || fn == nullptr) {
        cudaGetLastError();
        return AR_ERR_CUDA;
      }
      g_encode = reinterpret_cast<EncodeTiled>(fn);
    }
    for (int type = AR_TYPE_F32; type <= AR_TYPE_F16; ++type)
      for (int i = 0; i < 10; ++i) {
        const bool pair = i >= 4;  // 16 and 32 tokens of one CTA, 64 to 256 of a pair
        const I8Tensor k = i8_tensor(type, 16 << (i / 2), pair, i % 2 != 0);
        if (cudaFuncSetAttribute(reinterpret_cast<const void *>(k.kernel),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) != cudaSuccess) {
          cudaGetLastError();
          return AR_ERR_CUDA;
        }
      }
    // Clusters of 1, 2 and 4 pairs that the device runs at a time: some SMs
    // have no partners left.
    int found[3];
    for (int i = 2; i >= 0; --i) {
      const I8Tensor k = i8_tensor(AR_TYPE_BF16, 256, true, false);
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>((sms >> (i + 1)) << (i + 1)), 1, 1);
      cfg.blockDim = dim3(static_cast<unsigned>(k.threads), 1, 1);
      cfg.dynamicSmemBytes = static_cast<size_t>(k.smem);
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2u << i;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      found[i] = 0;
      if (cudaOccupancyMaxActiveClusters(&found[i], k.kernel, &cfg) != cudaSuccess || found[i] < 1) {
        cudaGetLastError();
        if (i == 0) return AR_ERR_CUDA;
        found[i] = 0;  // no splits into so many
      }
    }
    for (int i = 2; i >= 0; --i) of_device[dev][i] = found[i];
  }
  *pairs = of_device[dev];
  return AR_OK;
}

// Rows of K bytes as boxes of `box` rows x 128 bytes, 128-byte swizzle.
static bool encode(CUtensorMap *map, const int8_t *p, int64_t K, int64_t rows, int box) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  const cuuint32_t boxes[2] = {kI8StepK, static_cast<cuuint32_t>(box)}, ones[2] = {1, 1};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(p), dims, strides, boxes,
                  ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launch_i8_tensor(const I8Args &a, const I8Plan &plan, int pairs, cudaStream_t stream) {
  const int tokens = plan.tokens, split = plan.split;
  const bool pair = plan.pair;
  const I8Tensor k = i8_tensor(a.out_type, tokens, pair, a.gated != 0);
  I8TensorArgs t;
  t.a = a;
  t.a.aligned = aligned16(a.out) && a.width * type_size(a.out_type) % 16 == 0;
  if (!encode(&t.w_map, a.w, a.K, a.N, 64) || !encode(&t.x_map, a.x, a.K, a.m, k.x_rows))
    return AR_ERR_CUDA;
  const int64_t channels = (a.gated ? 64 : 128) * (pair ? 2 : 1);
  const int64_t tiles_n = (a.width + channels - 1) / channels, tiles_m = (a.m + tokens - 1) / tokens;
  t.tiles_n = static_cast<int>(tiles_n);
  t.tiles_m = static_cast<int>(tiles_m);
  t.split = split;
  t.group = 8;
  t.wait_limit_ns = kWaitLimitNs;
  const int64_t tiles = tiles_n * tiles_m;
  // Pairs without a split take tiles in turn.
  const int64_t grid = pair ? (split > 1 || tiles < pairs ? tiles : pairs) * split * 2 : tiles * split;
  if (grid > INT32_MAX) return AR_ERR_UNSUPPORTED;
  return launch_pdl(k.kernel, t, grid, k.threads, static_cast<size_t>(k.smem),
                    pair ? split * 2 : split, stream) == cudaSuccess
             ? AR_OK
             : AR_ERR_CUDA;
}

}  // namespace arn
