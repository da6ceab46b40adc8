// The tensor-core products' tensor maps and launches (i8_tensor.cuh).
#include <cstdlib>
#include <cstring>
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

int launch_i8_tensor(const I8Args &a, const I8Plan &plan, int pairs, cudaStream_t stream,
                     const I8Waits *waits) {
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
  t.waits = waits != nullptr ? *waits : I8Waits{kWaitLimitNs, kWaitLimitNs, -1, kI8AllStages};
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

using namespace arn;

namespace {

// Memory of the self-test, freed with it.
struct TestArray {
  void *p = nullptr;
  ~TestArray() {
    if (p) cudaFree(p);
  }
  bool make(size_t bytes, const void *from) {
    return cudaMalloc(&p, bytes) == cudaSuccess &&
           cudaMemcpy(p, from, bytes, cudaMemcpyHostToDevice) == cudaSuccess;
  }
};

constexpr int kTestM = 300, kTestN = 600, kTestK = 4096, kTestOuts = kTestM * kTestN;

// One shape: its outputs, then a run for each way of stopping, each followed by
// a run that has to give the same outputs again.  An AR_* status.
int selftest_shape(const I8Args &a, const I8Plan &plan, int device, const I8Waits &waits, float *want,
                   float *got) {
  const size_t bytes = static_cast<size_t>(kTestM) * a.width * sizeof(float);
  int st = launch_i8_tensor(a, plan, 1, nullptr);  // one pair takes all tiles
  if (st == AR_OK && cudaMemcpy(want, a.out, bytes, cudaMemcpyDeviceToHost) != cudaSuccess) st = AR_ERR_CUDA;
  if (st != AR_OK) return st;
  const int ranks = plan.split * (plan.pair ? 2 : 1);
  for (int rank = -1; rank < ranks; ++rank)
    for (int after = 0; after <= 2; after += 2) {
      I8Waits w = waits;
      w.stop_rank = rank;
      w.stop_after = after;
      st = launch_i8_tensor(a, plan, 1, nullptr, &w);
      if (st != AR_OK) return st;
      st = ar_device_status(device, 1);
      if (st != AR_ERR_TIMEOUT) return st == AR_OK ? AR_ERR_CUDA : st;
      st = launch_i8_tensor(a, plan, 1, nullptr);
      if (st == AR_OK && cudaMemcpy(got, a.out, bytes, cudaMemcpyDeviceToHost) != cudaSuccess)
        st = AR_ERR_CUDA;
      if (st == AR_OK) st = ar_device_status(device, 0);
      if (st == AR_OK && std::memcmp(want, got, bytes) != 0) st = AR_ERR_CUDA;
      if (st != AR_OK) return st;
    }
  return AR_OK;
}

int selftest_waits(int device, uint64_t limit_ns, int8_t *bytes, float *want, float *got) {
  int st = AR_OK;
  DeviceState *d = current_device(&st);
  const int *pairs = nullptr;
  if (d) st = ready_i8_tensor(d->sms, &pairs);
  if (st == AR_OK) st = ar_device_status(device, 0);
  if (st != AR_OK) return st;
  for (int i = 0; i < kTestN * kTestK; ++i) bytes[i] = static_cast<int8_t>(i % 251 * 37 % 255 - 127);
  for (int i = 0; i < kTestN; ++i) want[i] = 0.001f * static_cast<float>(1 + i % 7);
  TestArray x, xs, w, ws, out;
  if (!x.make(kTestM * kTestK, bytes) || !w.make(kTestN * kTestK, bytes) || !xs.make(kTestM * 4, want) ||
      !ws.make(kTestN * 4, want) || !out.make(kTestOuts * 4, want))
    return AR_ERR_CUDA;
  I8Args a = {};
  a.x = static_cast<const int8_t *>(x.p);
  a.xs = static_cast<const float *>(xs.p);
  a.w = static_cast<const int8_t *>(w.p);
  a.ws = static_cast<const float *>(ws.p);
  a.out = out.p;
  a.m = kTestM;
  a.N = kTestN;
  a.K = kTestK;
  a.out_type = AR_TYPE_F32;
  a.status = d->status;
  const I8Waits waits = {limit_ns, 10 * limit_ns, -1, 0};
  const I8Plan plans[] = {{16, 1, false}, {16, 4, false}, {32, 1, false}, {32, 8, false}, {64, 1, true},
                          {64, 2, true},  {128, 1, true}, {128, 4, true}, {256, 1, true}, {256, 4, true}};
  for (const I8Plan &p : plans) {
    if (p.pair && p.split > 1 && pairs[p.split == 2 ? 1 : 2] == 0) continue;  // such clusters do not fit
    for (a.gated = 0; a.gated < 2; ++a.gated) {
      a.width = a.gated ? kTestN / 2 : kTestN;
      st = selftest_shape(a, p, device, waits, want, got);
      if (st != AR_OK) return st;
    }
  }
  return AR_OK;
}

}  // namespace

extern "C" {

int ar_selftest_i8_waits(int device, unsigned limit_us) {
  if (device < 0 || device >= kMaxDevices || limit_us == 0 || limit_us > 100000u) return AR_ERR_ARG;
  int prev = -1;
  if (cudaGetDevice(&prev) != cudaSuccess || cudaSetDevice(device) != cudaSuccess) {
    cudaGetLastError();
    return AR_ERR_CUDA;
  }
  int8_t *bytes = static_cast<int8_t *>(std::malloc(kTestN * kTestK));
  float *outs = static_cast<float *>(std::calloc(2 * kTestOuts, sizeof(float)));
  const int st = bytes != nullptr && outs != nullptr
                     ? selftest_waits(device, static_cast<uint64_t>(limit_us) * 1000u, bytes, outs, outs + kTestOuts)
                     : AR_ERR_CUDA;
  std::free(bytes);
  std::free(outs);
  if (st == AR_ERR_CUDA) cudaGetLastError();
  cudaSetDevice(prev);
  return st;
}

}  // extern "C"
