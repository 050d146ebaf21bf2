// api.cu -- the extern "C" boundary of libfme.so (declared in include/fme.h):
// host-side argument checks, device checks, TMA descriptor encoding, launches.
// Nothing here allocates device memory or synchronises a stream, except
// fme_read_device_status, which is documented to synchronise.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

#include "../../include/fme.h"
#include "fme_launch.h"

namespace {

thread_local std::string g_last_cuda_error;

fme_status cuda_fail(cudaError_t err, const char *where) {
  g_last_cuda_error = std::string(where) + ": " + cudaGetErrorString(err);
  return FME_ERR_CUDA;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Device facts, looked up once per device.
struct DeviceInfo {
  std::atomic<int> state{0};  // 0 unknown, 1 supported, 2 unsupported
  int num_sms = 0;
};
DeviceInfo g_devices[64];
std::mutex g_device_mutex;

fme_status current_device(int *num_sms) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return cuda_fail(err, "cudaGetDevice");
  if (dev < 0 || dev >= 64) return FME_ERR_UNSUPPORTED_DEVICE;
  DeviceInfo &d = g_devices[dev];
  if (d.state.load(std::memory_order_acquire) == 0) {
    std::lock_guard<std::mutex> lock(g_device_mutex);
    if (d.state.load(std::memory_order_relaxed) == 0) {
      int major = 0, minor = 0, sms = 0;
      if ((err = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
          (err = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
          (err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return cuda_fail(err, "cudaDeviceGetAttribute");
      d.num_sms = sms;
      d.state.store((major == 10 && minor == 3) ? 1 : 2, std::memory_order_release);
    }
  }
  if (d.state.load(std::memory_order_acquire) != 1) return FME_ERR_UNSUPPORTED_DEVICE;
  *num_sms = d.num_sms;
  return FME_OK;
}

// cuTensorMapEncodeTiled from the driver, fetched once through the runtime.
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::once_flag g_encode_once;
EncodeTiledFn g_encode = nullptr;

fme_status get_encoder(EncodeTiledFn *fn) {
  std::call_once(g_encode_once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<EncodeTiledFn>(p);
  });
  if (g_encode == nullptr) {
    g_last_cuda_error = "cuTensorMapEncodeTiled not available from the driver";
    return FME_ERR_CUDA;
  }
  *fn = g_encode;
  return FME_OK;
}

// Encodes a map.  The encoder is a driver call and wants a current context, which a host thread that has made no
// runtime call yet does not have: the runtime binds the device's own, and the map is encoded again.
fme_status encode_map(const char *what, CUtensorMap *map, CUtensorMapDataType type, cuuint32_t rank, void *base,
                      const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box,
                      CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promotion) {
  EncodeTiledFn fn;
  const fme_status st = get_encoder(&fn);
  if (st != FME_OK) return st;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = CUDA_SUCCESS;
  for (int tries = 0; tries < 2; ++tries) {
    r = fn(map, type, rank, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_ERROR_INVALID_CONTEXT || tries > 0) break;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaSetDevice(dev);
    if (err != cudaSuccess) return cuda_fail(err, "cudaSetDevice");
  }
  if (r != CUDA_SUCCESS) {
    char buf[96];
    std::snprintf(buf, sizeof buf, "cuTensorMapEncodeTiled%s failed (CUresult %d)", what, static_cast<int>(r));
    g_last_cuda_error = buf;
    return FME_ERR_CUDA;
  }
  return FME_OK;
}

// 2-D uint8 tensor [rows x inner] (row stride `stride` bytes), box {128 bytes, box_rows},
// 128-byte swizzle, zero fill out of bounds.
fme_status encode_u8_2d(CUtensorMap *map, const void *base, uint64_t inner, uint64_t rows, uint64_t stride,
                        uint32_t box_rows) {
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {stride};
  cuuint32_t box[2] = {128, box_rows};
  return encode_map("", map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// bf16 matrix [rows x cols] (row stride cols * 2 bytes) for bulk tensor stores of
// 32 x 32 boxes with the 64-byte swizzle.  kWide..: boxes of 32 rows x 128 bytes with the
// 128-byte swizzle, bf16 or fp32.
enum class OutBox { kBf16, kWideBf16, kWideFp32 };
fme_status encode_bf16_out(CUtensorMap *map, void *base, uint64_t cols, uint64_t rows, OutBox kind = OutBox::kBf16) {
  const bool fp32 = kind == OutBox::kWideFp32, wide = kind != OutBox::kBf16;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * (fp32 ? 4 : 2)};
  cuuint32_t box[2] = {kind == OutBox::kWideBf16 ? 64u : 32u, 32};
  return encode_map(" (output)", map, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                    base, dims, strides, box, wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

// Tiled scales of a tensor as a 2-D map of 8-byte words: one row per 128-row
// block (`row_bytes` bytes each), boxes of `box_tiles` 512-byte tiles x `box_rows`
// blocks, no swizzle, zero fill out of bounds.
fme_status encode_scales_2d(CUtensorMap *map, const void *base, uint64_t row_blocks, uint64_t row_bytes,
                            uint32_t box_tiles, uint32_t box_rows) {
  cuuint64_t dims[2] = {row_bytes / 8, row_blocks};
  cuuint64_t strides[1] = {row_bytes};
  cuuint32_t box[2] = {64 * box_tiles, box_rows};
  return encode_map(" (scales)", map, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, const_cast<void *>(base), dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

int64_t padded_rows_bound(int64_t rows, int32_t groups) {
  if (rows < 0 || groups < 1) return 0;
  return ((rows + 127 * static_cast<int64_t>(groups)) / 128) * 128;
}

fme_status check_groups(int32_t num_groups) {
  return (num_groups < 1 || num_groups > FME_MAX_GROUPS) ? FME_ERR_INVALID_ARGUMENT : FME_OK;
}

}  // namespace

extern "C" {

int64_t fme_sf_padded_rows(int64_t rows, int32_t num_groups) { return padded_rows_bound(rows, num_groups); }

int64_t fme_sf_bytes(int64_t rows, int64_t cols, int32_t block, int32_t num_groups) {
  if (cols < 0 || block <= 0 || cols % block) return 0;
  const int64_t c4 = ((cols / block) + 3) / 4 * 4;
  return padded_rows_bound(rows, num_groups) * c4;
}

int64_t fme_colwise_ld(int64_t rows, int32_t num_groups) { return padded_rows_bound(rows, num_groups); }

int64_t fme_route_workspace_bytes(int64_t tokens, int32_t top_k, int32_t num_experts) {
  if (tokens < 0 || top_k < 1 || num_experts < 1) return 0;
  const int64_t chunks = (tokens * top_k + fme::kRouteChunkHost - 1) / fme::kRouteChunkHost;
  const int64_t b = chunks * num_experts * 4;
  return b < 16 ? 16 : b;
}

const char *fme_version(void) { return "fme 0.1.0 (sm_103a)"; }

const char *fme_last_cuda_error(void) { return g_last_cuda_error.c_str(); }

const char *fme_error_string(fme_status status) {
  switch (status) {
    case FME_OK: return "ok";
    case FME_ERR_INVALID_ARGUMENT: return "invalid argument";
    case FME_ERR_MISALIGNED: return "pointer or leading dimension not 16-byte aligned";
    case FME_ERR_UNSUPPORTED_SHAPE: return "shape outside the supported tiling";
    case FME_ERR_UNSUPPORTED_DEVICE: return "device is not compute capability 10.3 (GB300)";
    case FME_ERR_CUDA: return "CUDA error";
    case FME_ERR_DEVICE_TIMEOUT: return "a kernel's bounded wait ran out";
    case FME_ERR_DEVICE_BAD_OFFSETS: return "offsets do not rise from 0 to rows";
    case FME_ERR_DEVICE_BAD_INDEX: return "an expert id or a row index out of range";
    default: return "unknown status";
  }
}

fme_status fme_read_device_status(const int32_t *dev_status, void *stream, int32_t *raw) {
  if (dev_status == nullptr) return FME_ERR_INVALID_ARGUMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t host = 0;
  cudaError_t err = cudaMemcpyAsync(&host, dev_status, sizeof host, cudaMemcpyDeviceToHost, s);
  if (err != cudaSuccess) return cuda_fail(err, "cudaMemcpyAsync(status)");
  err = cudaStreamSynchronize(s);
  if (err != cudaSuccess) return cuda_fail(err, "cudaStreamSynchronize");
  if (raw) *raw = host;
  if (host & FME_DEV_BAD_OFFSETS) return FME_ERR_DEVICE_BAD_OFFSETS;
  if (host & FME_DEV_BAD_INDEX) return FME_ERR_DEVICE_BAD_INDEX;
  if (host & FME_DEV_TIMEOUT) return FME_ERR_DEVICE_TIMEOUT;
  return FME_OK;
}

fme_status quantize_nvfp4_pertoken(const void *x, int64_t rows, int64_t k, const int32_t *offsets,
                                   int32_t num_groups, uint8_t *codes, uint8_t *sf, float *row_scale,
                                   int32_t *dev_status, void *stream) {
  if (rows < 0 || check_groups(num_groups) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (offsets == nullptr && num_groups != 1) return FME_ERR_INVALID_ARGUMENT;
  if (k % 64 != 0 || k < 64 || k > 8192) return FME_ERR_UNSUPPORTED_SHAPE;
  if (rows > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return FME_OK;
  if (!x || !codes || !sf || !row_scale) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(sf) || !aligned16(row_scale)) return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchNvfp4 a{x, rows, k, offsets, num_groups, codes, sf, row_scale, dev_status, sms,
                     static_cast<cudaStream_t>(stream)};
  cudaError_t err = fme::launch_quantize_nvfp4(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "quantize_nvfp4_pertoken launch");
}

fme_status quantize_nvfp4_pertensor(const void *x, int64_t rows, int64_t k, const int32_t *offsets,
                                    int32_t num_groups, uint8_t *codes, uint8_t *sf, float *row_scale,
                                    float *tensor_amax, int32_t *dev_status, void *stream) {
  if (rows < 0 || check_groups(num_groups) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (offsets == nullptr && num_groups != 1) return FME_ERR_INVALID_ARGUMENT;
  if (k % 64 != 0 || k < 64 || k > 8192) return FME_ERR_UNSUPPORTED_SHAPE;
  if (rows > (int64_t(1) << 31) - 1 - 128 * static_cast<int64_t>(num_groups)) return FME_ERR_UNSUPPORTED_SHAPE;
  if (!tensor_amax) return FME_ERR_INVALID_ARGUMENT;
  if (rows > 0 && (!x || !codes || !sf || !row_scale)) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(sf) || !aligned16(row_scale) || !aligned16(tensor_amax))
    return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchNvfp4 a{x, rows, k, offsets, num_groups, codes, sf, row_scale, dev_status, sms,
                     static_cast<cudaStream_t>(stream)};
  cudaError_t err = fme::launch_quantize_nvfp4_pertensor(a, tensor_amax);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "quantize_nvfp4_pertensor launch");
}

fme_status swiglu_quantize_nvfp4(const void *gate_up, int64_t rows, int64_t inter, const int32_t *offsets,
                                 int32_t num_groups, uint8_t *codes, uint8_t *sf, float *row_scale, void *h,
                                 int32_t *dev_status, void *stream) {
  if (rows < 0 || check_groups(num_groups) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (offsets == nullptr && num_groups != 1) return FME_ERR_INVALID_ARGUMENT;
  if (inter % 64 != 0 || inter < 64 || inter > 8192) return FME_ERR_UNSUPPORTED_SHAPE;
  if (rows > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return FME_OK;
  if (!gate_up || !codes || !sf || !row_scale) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(gate_up) || !aligned16(codes) || !aligned16(sf) || !aligned16(row_scale) || !aligned16(h))
    return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchNvfp4 a{gate_up, rows, inter, offsets, num_groups, codes, sf, row_scale, dev_status, sms,
                     static_cast<cudaStream_t>(stream)};
  a.swiglu = true;
  a.h_out = h;
  cudaError_t err = fme::launch_quantize_nvfp4(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "swiglu_quantize_nvfp4 launch");
}

fme_status moe_route(const int32_t *topk_ids, int64_t tokens, int32_t top_k, int32_t num_experts, int32_t *offsets,
                     int32_t *row_of, int32_t *src_row, void *workspace, int64_t workspace_bytes,
                     int32_t *dev_status, void *stream) {
  if (tokens < 0 || top_k < 1 || top_k > 64 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (tokens * top_k > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  if (!offsets || !workspace) return FME_ERR_INVALID_ARGUMENT;
  if (tokens > 0 && (!topk_ids || !row_of || !src_row)) return FME_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < fme_route_workspace_bytes(tokens, top_k, num_experts)) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(topk_ids) || !aligned16(offsets) || !aligned16(row_of) || !aligned16(src_row) ||
      !aligned16(workspace))
    return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchRoute r{topk_ids, tokens, top_k, num_experts, offsets, row_of, src_row,
                     static_cast<int32_t *>(workspace), dev_status, static_cast<cudaStream_t>(stream)};
  cudaError_t err = fme::launch_route(r);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "moe_route launch");
}

fme_status moe_route_noalloc(const int32_t *topk_ids, int64_t tokens, int32_t top_k, int32_t num_experts,
                             int32_t *offsets, int32_t *row_of, int32_t *src_row, int32_t *dev_status,
                             void *stream) {
  if (tokens < 0 || top_k < 1 || top_k > 64 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (tokens * top_k > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  const int64_t chunks = (tokens * top_k + fme::kRouteChunkHost - 1) / fme::kRouteChunkHost;
  if (chunks * num_experts > fme::kRouteStaticWords) return FME_ERR_UNSUPPORTED_SHAPE;
  if (!offsets) return FME_ERR_INVALID_ARGUMENT;
  if (tokens > 0 && (!topk_ids || !row_of || !src_row)) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(topk_ids) || !aligned16(offsets) || !aligned16(row_of) || !aligned16(src_row))
    return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchRoute r{topk_ids, tokens, top_k, num_experts, offsets, row_of, src_row, nullptr, dev_status,
                     static_cast<cudaStream_t>(stream)};
  cudaError_t err = fme::launch_route_static(r);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "moe_route_noalloc launch");
}

fme_status permute_quantize_nvfp4(const void *x, int64_t tokens, int64_t k, const int32_t *src_row, int32_t top_k,
                                  const int32_t *offsets, int32_t num_experts, uint8_t *codes, uint8_t *sf,
                                  float *row_scale, int32_t *dev_status, void *stream) {
  if (tokens < 0 || top_k < 1 || top_k > 64 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (k % 64 != 0 || k < 64 || k > 8192) return FME_ERR_UNSUPPORTED_SHAPE;
  const int64_t rows = tokens * top_k;
  if (rows > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  if (!offsets) return FME_ERR_INVALID_ARGUMENT;
  if (rows == 0) return FME_OK;
  if (!x || !src_row || !codes || !sf || !row_scale) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(src_row) || !aligned16(codes) || !aligned16(sf) || !aligned16(row_scale) ||
      !aligned16(offsets))
    return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchNvfp4 a{x, rows, k, offsets, num_experts, codes, sf, row_scale, dev_status, sms,
                     static_cast<cudaStream_t>(stream)};
  a.gather = src_row;
  a.gather_div = top_k;
  a.gather_limit = tokens;
  cudaError_t err = fme::launch_quantize_nvfp4(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "permute_quantize_nvfp4 launch");
}

fme_status permute_quantize_mxfp8(const void *x, int64_t tokens, int64_t k, const int32_t *src_row, int32_t top_k,
                                  const int32_t *offsets, int32_t num_experts, uint8_t *codes, uint8_t *sf,
                                  int32_t *dev_status, void *stream) {
  if (tokens < 0 || top_k < 1 || top_k > 64 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (k % 32 != 0 || k < 32 || k > 65536) return FME_ERR_UNSUPPORTED_SHAPE;
  const int64_t rows = tokens * top_k;
  if (rows > (int64_t(1) << 31) - 1 - 128 * static_cast<int64_t>(num_experts)) return FME_ERR_UNSUPPORTED_SHAPE;
  if (!offsets) return FME_ERR_INVALID_ARGUMENT;
  if (rows == 0) return FME_OK;
  if (!x || !src_row || !codes || !sf) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(src_row) || !aligned16(codes) || !aligned16(sf)) return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchMxfp8 a{x, rows, k, offsets, num_experts, codes, sf, nullptr, 0, dev_status, sms,
                     static_cast<cudaStream_t>(stream)};
  a.gather = src_row;
  a.gather_div = top_k;
  a.gather_limit = tokens;
  cudaError_t err = fme::launch_quantize_mxfp8_rows(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "permute_quantize_mxfp8 launch");
}

fme_status moe_combine(const void *y, int64_t rows_y, const int32_t *row_of, const float *weights, int64_t tokens,
                       int32_t top_k, int64_t n, void *out, int32_t *dev_status, void *stream) {
  if (tokens < 0 || rows_y < 0 || top_k < 1 || top_k > 64 || n < 0) return FME_ERR_INVALID_ARGUMENT;
  if (n % 8 != 0 || n == 0 || n > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  if (tokens * top_k > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  if (tokens == 0) return FME_OK;
  if (!row_of || !weights || !out || (rows_y > 0 && !y)) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(y) || !aligned16(row_of) || !aligned16(weights) || !aligned16(out)) return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchCombine c{y, row_of, weights, tokens, top_k, n, rows_y, out, dev_status, sms,
                       static_cast<cudaStream_t>(stream)};
  cudaError_t err = fme::launch_combine(c);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "moe_combine launch");
}

fme_status quantize_mxfp8(const void *x, int64_t rows, int64_t cols, int32_t axis, const int32_t *offsets,
                          int32_t num_groups, uint8_t *codes, uint8_t *sf, int32_t *padded_offsets,
                          int32_t *dev_status, void *stream) {
  const bool ceil_scale = (axis & FME_MX_SCALE_CEIL) != 0;
  axis &= ~FME_MX_SCALE_CEIL;
  if (rows < 0 || check_groups(num_groups) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (offsets == nullptr && num_groups != 1) return FME_ERR_INVALID_ARGUMENT;
  if (axis != FME_ROWWISE && axis != FME_COLWISE) return FME_ERR_INVALID_ARGUMENT;
  if (rows > (int64_t(1) << 31) - 1 - 128 * static_cast<int64_t>(num_groups)) return FME_ERR_UNSUPPORTED_SHAPE;
  if (axis == FME_ROWWISE) {
    if (padded_offsets != nullptr) return FME_ERR_INVALID_ARGUMENT;
    if (cols % 32 != 0 || cols < 32 || cols > 65536) return FME_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return FME_OK;
  } else {
    if (cols % 128 != 0 || cols < 128 || cols > 65536) return FME_ERR_UNSUPPORTED_SHAPE;
    if (padded_offsets == nullptr) return FME_ERR_INVALID_ARGUMENT;
    if (!aligned16(padded_offsets)) return FME_ERR_MISALIGNED;
  }
  if ((!x && rows > 0) || !codes || !sf) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(sf)) return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchMxfp8 a{x, rows, cols, offsets, num_groups, codes, sf, padded_offsets,
                     fme_colwise_ld(rows, num_groups), dev_status, sms, static_cast<cudaStream_t>(stream)};
  a.ceil_scale = ceil_scale;
  cudaError_t err =
      (axis == FME_ROWWISE) ? fme::launch_quantize_mxfp8_rows(a) : fme::launch_quantize_mxfp8_cols(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "quantize_mxfp8 launch");
}

fme_status quantize_mxfp8_rowcol(const void *x, int64_t rows, int64_t cols, const int32_t *offsets,
                                 int32_t num_groups, uint8_t *row_codes, uint8_t *row_sf, uint8_t *col_codes,
                                 uint8_t *col_sf, int32_t *padded_offsets, int32_t *dev_status, void *stream) {
  if (rows < 0 || check_groups(num_groups) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (offsets == nullptr && num_groups != 1) return FME_ERR_INVALID_ARGUMENT;
  if (rows > (int64_t(1) << 31) - 1 - 128 * static_cast<int64_t>(num_groups)) return FME_ERR_UNSUPPORTED_SHAPE;
  if (cols % 128 != 0 || cols < 128 || cols > 65536) return FME_ERR_UNSUPPORTED_SHAPE;
  if (!padded_offsets || !col_codes || !col_sf || !row_sf || (rows > 0 && (!x || !row_codes)))
    return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(row_codes) || !aligned16(row_sf) || !aligned16(col_codes) || !aligned16(col_sf) ||
      !aligned16(padded_offsets))
    return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchMxfp8 a{x, rows, cols, offsets, num_groups, col_codes, col_sf, padded_offsets,
                     fme_colwise_ld(rows, num_groups), dev_status, sms, static_cast<cudaStream_t>(stream)};
  cudaError_t err = fme::launch_quantize_mxfp8_rowcol(a, row_codes, row_sf);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "quantize_mxfp8_rowcol launch");
}

fme_status swiglu_backward_quantize_mxfp8(const void *gate_up, const void *dh, int64_t rows, int64_t inter,
                                          const int32_t *offsets, int32_t num_groups, uint8_t *row_codes,
                                          uint8_t *row_sf, uint8_t *col_codes, uint8_t *col_sf,
                                          int32_t *padded_offsets, void *d_gate_up, int32_t *dev_status,
                                          void *stream) {
  if (rows < 0 || check_groups(num_groups) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (offsets == nullptr && num_groups != 1) return FME_ERR_INVALID_ARGUMENT;
  if (rows > (int64_t(1) << 31) - 1 - 128 * static_cast<int64_t>(num_groups)) return FME_ERR_UNSUPPORTED_SHAPE;
  if (inter % 128 != 0 || inter < 128 || inter > 32768) return FME_ERR_UNSUPPORTED_SHAPE;
  if (!padded_offsets || !col_codes || !col_sf || !row_sf || (rows > 0 && (!gate_up || !dh || !row_codes)))
    return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(gate_up) || !aligned16(dh) || !aligned16(row_codes) || !aligned16(row_sf) ||
      !aligned16(col_codes) || !aligned16(col_sf) || !aligned16(padded_offsets) || !aligned16(d_gate_up))
    return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchMxfp8 a{gate_up, rows, 2 * inter, offsets, num_groups, col_codes, col_sf, padded_offsets,
                     fme_colwise_ld(rows, num_groups), dev_status, sms, static_cast<cudaStream_t>(stream)};
  a.dh = dh;
  a.d_out = d_gate_up;
  cudaError_t err = fme::launch_swiglu_bwd_mxfp8(a, row_codes, row_sf);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "swiglu_backward_quantize_mxfp8 launch");
}

// The NVFP4 forward, plain (y [m x n]) or with the SwiGLU epilogue (y = h [m x n / 2]).
static fme_status fwd_nvfp4(bool swiglu, const uint8_t *a_codes, const uint8_t *a_sf, const float *a_scale,
                            const uint8_t *b_codes, const uint8_t *b_sf, const float *b_scale, const int32_t *offsets,
                            int32_t num_experts, int64_t m, int64_t n, int64_t k, void *y, int32_t *dev_status,
                            void *stream) {
  if (m < 0 || n < 0 || k < 0 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (n % 256 != 0 || n == 0 || k % 256 != 0 || k == 0 || k > 65536) return FME_ERR_UNSUPPORTED_SHAPE;
  if (m > (int64_t(1) << 31) - 1 || static_cast<int64_t>(num_experts) * n > (int64_t(1) << 31) - 1)
    return FME_ERR_UNSUPPORTED_SHAPE;
  if (!offsets) return FME_ERR_INVALID_ARGUMENT;
  if (m == 0) return FME_OK;
  if (!a_codes || !a_sf || !a_scale || !b_codes || !b_sf || !b_scale || !y) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(a_codes) || !aligned16(a_sf) || !aligned16(a_scale) || !aligned16(b_codes) ||
      !aligned16(b_sf) || !aligned16(b_scale) || !aligned16(y) || !aligned16(offsets))
    return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchGemm a{};
  a.kind = swiglu ? fme::GemmKind::kFwdNvfp4Swiglu : fme::GemmKind::kFwdNvfp4;
  if ((st = encode_u8_2d(&a.map_a, a_codes, k / 2, m, k / 2, 128)) != FME_OK) return st;
  if ((st = encode_u8_2d(&a.map_b, b_codes, k / 2, static_cast<uint64_t>(num_experts) * n, k / 2, 128)) != FME_OK)
    return st;
  // scales: (k / 64) tiles of 512 bytes per 128-row block; a stage takes 4 tiles
  if ((st = encode_scales_2d(&a.map_sfa, a_sf, padded_rows_bound(m, num_experts) / 128, (k / 64) * 512, 4, 1)) !=
      FME_OK)
    return st;
  // B scales: the same tiled layout (the stacked weights are one group of
  // num_experts * n rows); a stage takes 4 tiles of each of the tile's two 128-row
  // blocks, adjacent (one copy) or, with SwiGLU, a gate and an up block (two copies)
  if ((st = encode_scales_2d(&a.map_sfb, b_sf, static_cast<uint64_t>(num_experts) * n / 128, (k / 64) * 512, 4,
                             swiglu ? 1 : 2)) != FME_OK)
    return st;
  if ((st = encode_bf16_out(&a.map_y, y, swiglu ? n / 2 : n, m)) != FME_OK) return st;
  a.a_scale = a_scale;
  a.b_scale = b_scale;
  a.offsets = offsets;
  a.num_experts = num_experts;
  a.m = m;
  a.n = n;
  a.k = k;
  a.y = y;
  a.status = dev_status;
  a.num_sms = sms;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_grouped_gemm(a);
  return err == cudaSuccess ? FME_OK
                            : cuda_fail(err, swiglu ? "grouped_gemm_fwd_nvfp4_swiglu launch" : "grouped_gemm_fwd_nvfp4 launch");
}

fme_status grouped_gemm_fwd_nvfp4(const uint8_t *a_codes, const uint8_t *a_sf, const float *a_scale,
                                  const uint8_t *b_codes, const uint8_t *b_sf, const float *b_scale,
                                  const int32_t *offsets, int32_t num_experts, int64_t m, int64_t n, int64_t k,
                                  void *y, int32_t *dev_status, void *stream) {
  return fwd_nvfp4(false, a_codes, a_sf, a_scale, b_codes, b_sf, b_scale, offsets, num_experts, m, n, k, y,
                   dev_status, stream);
}

fme_status grouped_gemm_fwd_nvfp4_swiglu(const uint8_t *a_codes, const uint8_t *a_sf, const float *a_scale,
                                         const uint8_t *b_codes, const uint8_t *b_sf, const float *b_scale,
                                         const int32_t *offsets, int32_t num_experts, int64_t m, int64_t n,
                                         int64_t k, void *h, int32_t *dev_status, void *stream) {
  return fwd_nvfp4(true, a_codes, a_sf, a_scale, b_codes, b_sf, b_scale, offsets, num_experts, m, n, k, h,
                   dev_status, stream);
}

fme_status grouped_gemm_fwd_mxfp8(const uint8_t *a_codes, const uint8_t *a_sf, const uint8_t *b_codes,
                                  const uint8_t *b_sf, const int32_t *offsets, int32_t num_experts, int64_t m,
                                  int64_t n, int64_t k, void *y, int32_t *dev_status, void *stream) {
  if (m < 0 || n < 0 || k < 0 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (n % 256 != 0 || n == 0 || k % 128 != 0 || k == 0 || k > 65536) return FME_ERR_UNSUPPORTED_SHAPE;
  if (m > (int64_t(1) << 31) - 1 || static_cast<int64_t>(num_experts) * n > (int64_t(1) << 31) - 1)
    return FME_ERR_UNSUPPORTED_SHAPE;
  if (!offsets) return FME_ERR_INVALID_ARGUMENT;
  if (m == 0) return FME_OK;
  if (!a_codes || !a_sf || !b_codes || !b_sf || !y) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(a_codes) || !aligned16(a_sf) || !aligned16(b_codes) || !aligned16(b_sf) || !aligned16(y) ||
      !aligned16(offsets))
    return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchGemm a{};
  a.kind = fme::GemmKind::kFwdMxfp8;
  if ((st = encode_u8_2d(&a.map_a, a_codes, k, m, k, 128)) != FME_OK) return st;
  if ((st = encode_u8_2d(&a.map_b, b_codes, k, static_cast<uint64_t>(num_experts) * n, k, 128)) != FME_OK)
    return st;
  // row-wise E8M0 scales: (k / 128) tiles of 512 bytes per 128-row block; a stage takes one
  if ((st = encode_scales_2d(&a.map_sfa, a_sf, padded_rows_bound(m, num_experts) / 128, (k / 128) * 512, 1, 1)) !=
      FME_OK)
    return st;
  if ((st = encode_scales_2d(&a.map_sfb, b_sf, static_cast<uint64_t>(num_experts) * n / 128, (k / 128) * 512, 1,
                             2)) != FME_OK)
    return st;
  if ((st = encode_bf16_out(&a.map_y, y, n, m)) != FME_OK) return st;
  a.offsets = offsets;
  a.num_experts = num_experts;
  a.m = m;
  a.n = n;
  a.k = k;
  a.y = y;
  a.status = dev_status;
  a.num_sms = sms;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_grouped_gemm(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "grouped_gemm_fwd_mxfp8 launch");
}

fme_status grouped_gemm_dgrad_mxfp8(const uint8_t *a_codes, const uint8_t *a_sf, const uint8_t *b_codes,
                                    const uint8_t *b_sf, int64_t ldb, const int32_t *offsets, int32_t num_experts,
                                    int64_t m, int64_t n, int64_t k, void *y, int32_t *dev_status, void *stream) {
  if (m < 0 || n < 0 || k < 0 || ldb < 0 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (n % 256 != 0 || n == 0 || k % 128 != 0 || k == 0 || ldb % 128 != 0) return FME_ERR_UNSUPPORTED_SHAPE;
  if (ldb < static_cast<int64_t>(num_experts) * k) return FME_ERR_INVALID_ARGUMENT;
  if (m > (int64_t(1) << 31) - 1 || ldb > (int64_t(1) << 31) - 1 || k > 65536) return FME_ERR_UNSUPPORTED_SHAPE;
  if (!offsets) return FME_ERR_INVALID_ARGUMENT;
  if (m == 0) return FME_OK;
  if (!a_codes || !a_sf || !b_codes || !b_sf || !y) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(a_codes) || !aligned16(a_sf) || !aligned16(b_codes) || !aligned16(b_sf) || !aligned16(y) ||
      !aligned16(offsets))
    return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchGemm a{};
  a.kind = fme::GemmKind::kDgradMxfp8;
  if ((st = encode_u8_2d(&a.map_a, a_codes, k, m, k, 128)) != FME_OK) return st;
  if ((st = encode_u8_2d(&a.map_b, b_codes, ldb, n, ldb, 128)) != FME_OK) return st;
  if ((st = encode_scales_2d(&a.map_sfa, a_sf, padded_rows_bound(m, num_experts) / 128, (k / 128) * 512, 1, 1)) !=
      FME_OK)
    return st;
  if ((st = encode_scales_2d(&a.map_sfb, b_sf, n / 128, (ldb / 128) * 512, 1, 2)) != FME_OK) return st;
  if ((st = encode_bf16_out(&a.map_y, y, n, m)) != FME_OK) return st;
  a.offsets = offsets;
  a.num_experts = num_experts;
  a.m = m;
  a.n = n;
  a.k = k;
  a.ldb = ldb;
  a.y = y;
  a.status = dev_status;
  a.num_sms = sms;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_grouped_gemm(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "grouped_gemm_dgrad_mxfp8 launch");
}

static fme_status wgrad_call(const uint8_t *a_codes, const uint8_t *a_sf, int64_t lda, const uint8_t *b_codes,
                             const uint8_t *b_sf, int64_t ldb, const int32_t *padded_offsets, int32_t num_experts,
                             int64_t m, int64_t n, void *y, bool accumulate, int32_t *dev_status, void *stream,
                             const char *what) {
  if (m < 0 || n < 0 || lda < 0 || ldb < 0 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (m % 256 != 0 || m == 0 || n % 256 != 0 || n == 0 || lda % 128 != 0 || ldb % 128 != 0)
    return FME_ERR_UNSUPPORTED_SHAPE;
  if (lda > (int64_t(1) << 31) - 1 || ldb > (int64_t(1) << 31) - 1 || m > 65536 || n > 65536)
    return FME_ERR_UNSUPPORTED_SHAPE;
  if (!padded_offsets || !y) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(y) || !aligned16(padded_offsets)) return FME_ERR_MISALIGNED;
  const bool has_positions = lda > 0 && ldb > 0;
  if (has_positions) {
    if (!a_codes || !a_sf || !b_codes || !b_sf) return FME_ERR_INVALID_ARGUMENT;
    if (!aligned16(a_codes) || !aligned16(a_sf) || !aligned16(b_codes) || !aligned16(b_sf))
      return FME_ERR_MISALIGNED;
  }
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchGemm a{};
  a.kind = fme::GemmKind::kWgradMxfp8;
  // With no positions at all every expert is empty: the maps are never used, so
  // point them at a small dummy extent of y (always at least 256 x 256 x 2 bytes).
  const void *abase = has_positions ? static_cast<const void *>(a_codes) : y;
  const void *bbase = has_positions ? static_cast<const void *>(b_codes) : y;
  const void *sabase = has_positions ? static_cast<const void *>(a_sf) : y;
  const void *sbbase = has_positions ? static_cast<const void *>(b_sf) : y;
  const int64_t lda_e = has_positions ? lda : 128, ldb_e = has_positions ? ldb : 128;
  if ((st = encode_u8_2d(&a.map_a, abase, lda_e, has_positions ? m : 128, lda_e, 128)) != FME_OK) return st;
  if ((st = encode_u8_2d(&a.map_b, bbase, ldb_e, has_positions ? n : 128, ldb_e, 128)) != FME_OK) return st;
  if ((st = encode_scales_2d(&a.map_sfa, sabase, has_positions ? m / 128 : 1, (lda_e / 128) * 512, 1, 1)) != FME_OK)
    return st;
  if ((st = encode_scales_2d(&a.map_sfb, sbbase, has_positions ? n / 128 : 2, (ldb_e / 128) * 512, 1, 2)) != FME_OK)
    return st;
  // dW [num_experts * m x n] bf16 for bulk stores (the fp32 accumulate writes with plain stores)
  if (!accumulate && (st = encode_bf16_out(&a.map_y, y, n, static_cast<uint64_t>(num_experts) * m)) != FME_OK)
    return st;
  a.offsets = padded_offsets;
  a.num_experts = num_experts;
  a.m = m;
  a.n = n;
  a.k = 0;
  a.lda = lda;
  a.ldb = ldb;
  a.y = y;
  a.accumulate = accumulate;
  a.status = dev_status;
  a.num_sms = sms;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_grouped_gemm(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, what);
}

fme_status grouped_gemm_wgrad_mxfp8(const uint8_t *a_codes, const uint8_t *a_sf, int64_t lda,
                                    const uint8_t *b_codes, const uint8_t *b_sf, int64_t ldb,
                                    const int32_t *padded_offsets, int32_t num_experts, int64_t m, int64_t n,
                                    void *y, int32_t *dev_status, void *stream) {
  return wgrad_call(a_codes, a_sf, lda, b_codes, b_sf, ldb, padded_offsets, num_experts, m, n, y, false, dev_status,
                    stream, "grouped_gemm_wgrad_mxfp8 launch");
}

fme_status grouped_gemm_wgrad_mxfp8_accumulate(const uint8_t *a_codes, const uint8_t *a_sf, int64_t lda,
                                               const uint8_t *b_codes, const uint8_t *b_sf, int64_t ldb,
                                               const int32_t *padded_offsets, int32_t num_experts, int64_t m,
                                               int64_t n, float *dw_acc, int32_t *dev_status, void *stream) {
  return wgrad_call(a_codes, a_sf, lda, b_codes, b_sf, ldb, padded_offsets, num_experts, m, n, dw_acc, true,
                    dev_status, stream, "grouped_gemm_wgrad_mxfp8_accumulate launch");
}

// ------------------------------------------------------------ FP8 block-128 --
namespace {

// Columns of an FP8 block-128 tensor: its code rows are a multiple of 16 bytes.
bool block128_cols(int64_t c) { return c >= 16 && c <= 65536 && c % 16 == 0; }

// 3-D uint8 weights [experts][n][k], box {128, 128, 1}, 128-byte swizzle, zero fill past each
// expert's n and k.
fme_status encode_u8_weights(CUtensorMap *map, const void *base, uint64_t experts, uint64_t n, uint64_t k) {
  cuuint64_t dims[3] = {k, n, experts};
  cuuint64_t strides[2] = {k, n * k};
  cuuint32_t box[3] = {128, 128, 1};
  return encode_map(" (weights)", map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// 128 x 128 tiles of a [rows x cols] tensor fit one launch.
bool tiles_fit(int64_t row_chunks, int64_t cols) {
  return row_chunks * ((cols + 127) / 128) <= (int64_t(1) << 31) - 1;
}

fme_status fp8_rows(const void *x, int64_t x_rows, int64_t rows, int64_t cols, const int32_t *src_row, int32_t top_k,
                    uint8_t *codes, float *scale, int32_t *dev_status, void *stream, const char *what) {
  if (!block128_cols(cols) || rows > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return FME_OK;
  if (!x || !codes || !scale) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scale) || !aligned16(src_row)) return FME_ERR_MISALIGNED;
  fme::LaunchFp8Quant a{};
  fme_status st = current_device(&a.num_sms);
  if (st != FME_OK) return st;
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.codes = codes;
  a.scale = scale;
  a.gather = src_row;
  a.gather_div = top_k;
  a.gather_limit = x_rows;
  a.status = dev_status;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_fp8_block128_rows(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, what);
}

fme_status fp8_cols(const void *x, int64_t rows, int64_t cols, const int32_t *offsets, int32_t num_groups,
                    uint8_t *row_codes, float *row_scale, uint8_t *codes, float *scale, int32_t *padded_offsets,
                    int32_t *dev_status, void *stream, const char *what) {
  const int64_t ld = fme_colwise_ld(rows, num_groups);
  if (!block128_cols(cols) || ld > (int64_t(1) << 31) - 1 || !tiles_fit(ld / 128, cols))
    return FME_ERR_UNSUPPORTED_SHAPE;
  if (!padded_offsets || (ld > 0 && (!codes || !scale)) || (rows > 0 && !x)) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scale) || !aligned16(row_codes) || !aligned16(row_scale) ||
      !aligned16(padded_offsets))
    return FME_ERR_MISALIGNED;
  fme::LaunchFp8Quant a{};
  fme_status st = current_device(&a.num_sms);
  if (st != FME_OK) return st;
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.offsets = offsets;
  a.num_groups = num_groups;
  a.codes = codes;
  a.scale = scale;
  a.padded_offsets = padded_offsets;
  a.ld = ld;
  a.row_codes = row_codes;
  a.row_scale = row_scale;
  a.status = dev_status;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_fp8_block128_cols(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, what);
}

// The forward (out = n columns, contraction k) and dgrad (out = k columns, contraction n).
fme_status block128_rows_gemm(bool dgrad, const uint8_t *a_codes, const float *a_scale, const uint8_t *w_codes,
                              const float *w_scale, const int32_t *offsets, int32_t num_experts, int64_t m, int64_t n,
                              int64_t k, void *y, int32_t *dev_status, void *stream, const char *what) {
  if (m < 0 || n < 0 || k < 0 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (!block128_cols(n) || !block128_cols(k)) return FME_ERR_UNSUPPORTED_SHAPE;
  // row coordinates of the last, partly empty tiles and the number of tiles stay in 32 bits
  if (m > (int64_t(1) << 31) - 1 - 256) return FME_ERR_UNSUPPORTED_SHAPE;
  if ((m / 64 + num_experts) * (((dgrad ? k : n) + 127) / 128) > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  if (!offsets) return FME_ERR_INVALID_ARGUMENT;
  if (m == 0) return FME_OK;
  if (!a_codes || !a_scale || !w_codes || !w_scale || !y) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(a_codes) || !aligned16(a_scale) || !aligned16(w_codes) || !aligned16(w_scale) || !aligned16(y) ||
      !aligned16(offsets))
    return FME_ERR_MISALIGNED;
  fme::LaunchBlock128 a{};
  fme_status st = current_device(&a.num_sms);
  if (st != FME_OK) return st;
  a.k = dgrad ? n : k;
  a.n = dgrad ? k : n;
  const bool few = !dgrad && fme::block128_few_rows(m, num_experts);
  CUtensorMap &rows_map = few ? a.map_b : a.map_a, &w_map = few ? a.map_a : a.map_b;
  if ((st = encode_u8_2d(&rows_map, a_codes, a.k, m, a.k, few ? 16 : 128)) != FME_OK) return st;
  if ((st = encode_u8_weights(&w_map, w_codes, num_experts, n, k)) != FME_OK) return st;
  if ((st = encode_bf16_out(&a.map_y, y, a.n, m, OutBox::kWideBf16)) != FME_OK) return st;
  a.a_scale = a_scale;
  a.b_scale = w_scale;
  a.offsets = offsets;
  a.num_experts = num_experts;
  a.m = m;
  a.y = y;
  a.status = dev_status;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = dgrad ? fme::launch_block128_dgrad(a) : fme::launch_block128_fwd(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, what);
}

}  // namespace

fme_status quantize_fp8_block128(const void *x, int64_t rows, int64_t cols, int32_t axis, const int32_t *offsets,
                                 int32_t num_groups, uint8_t *codes, float *scale, int32_t *padded_offsets,
                                 int32_t *dev_status, void *stream) {
  if (rows < 0 || cols < 0 || check_groups(num_groups) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (offsets == nullptr && num_groups != 1) return FME_ERR_INVALID_ARGUMENT;
  if (axis == FME_ROWWISE) {
    if (padded_offsets != nullptr) return FME_ERR_INVALID_ARGUMENT;
    return fp8_rows(x, rows, rows, cols, nullptr, 1, codes, scale, dev_status, stream, "quantize_fp8_block128 launch");
  }
  if (axis != FME_COLWISE) return FME_ERR_INVALID_ARGUMENT;
  return fp8_cols(x, rows, cols, offsets, num_groups, nullptr, nullptr, codes, scale, padded_offsets, dev_status,
                  stream, "quantize_fp8_block128 launch");
}

fme_status quantize_fp8_block128_rowcol(const void *x, int64_t rows, int64_t cols, const int32_t *offsets,
                                        int32_t num_groups, uint8_t *row_codes, float *row_scale, uint8_t *col_codes,
                                        float *col_scale, int32_t *padded_offsets, int32_t *dev_status,
                                        void *stream) {
  if (rows < 0 || cols < 0 || check_groups(num_groups) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (offsets == nullptr && num_groups != 1) return FME_ERR_INVALID_ARGUMENT;
  if (rows > 0 && (!row_codes || !row_scale)) return FME_ERR_INVALID_ARGUMENT;
  return fp8_cols(x, rows, cols, offsets, num_groups, rows > 0 ? row_codes : nullptr, row_scale, col_codes, col_scale,
                  padded_offsets, dev_status, stream, "quantize_fp8_block128_rowcol launch");
}

fme_status permute_quantize_fp8_block128(const void *x, int64_t tokens, int64_t cols, const int32_t *src_row,
                                         int32_t top_k, uint8_t *codes, float *scale, int32_t *dev_status,
                                         void *stream) {
  if (tokens < 0 || cols < 0 || top_k < 1 || top_k > 64) return FME_ERR_INVALID_ARGUMENT;
  if (tokens > 0 && !src_row) return FME_ERR_INVALID_ARGUMENT;
  return fp8_rows(x, tokens, tokens * top_k, cols, src_row, top_k, codes, scale, dev_status, stream,
                  "permute_quantize_fp8_block128 launch");
}

fme_status quantize_fp8_block128_weights(const void *w, int32_t num_experts, int64_t n, int64_t k, uint8_t *codes,
                                         float *scale, void *stream) {
  if (n < 0 || k < 0 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (!block128_cols(n) || !block128_cols(k) || !tiles_fit(num_experts * ((n + 127) / 128), k))
    return FME_ERR_UNSUPPORTED_SHAPE;
  if (!w || !codes || !scale) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(w) || !aligned16(codes) || !aligned16(scale)) return FME_ERR_MISALIGNED;
  fme::LaunchFp8Quant a{};
  fme_status st = current_device(&a.num_sms);
  if (st != FME_OK) return st;
  a.x = w;
  a.rows = n;
  a.cols = k;
  a.num_groups = num_experts;
  a.codes = codes;
  a.scale = scale;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_fp8_block128_weights(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "quantize_fp8_block128_weights launch");
}

fme_status grouped_gemm_fwd_fp8_block128(const uint8_t *a_codes, const float *a_scale, const uint8_t *w_codes,
                                         const float *w_scale, const int32_t *offsets, int32_t num_experts, int64_t m,
                                         int64_t n, int64_t k, void *y, int32_t *dev_status, void *stream) {
  return block128_rows_gemm(false, a_codes, a_scale, w_codes, w_scale, offsets, num_experts, m, n, k, y, dev_status,
                            stream, "grouped_gemm_fwd_fp8_block128 launch");
}

fme_status grouped_gemm_dgrad_fp8_block128(const uint8_t *dy_codes, const float *dy_scale, const uint8_t *w_codes,
                                           const float *w_scale, const int32_t *offsets, int32_t num_experts,
                                           int64_t m, int64_t n, int64_t k, void *dx, int32_t *dev_status,
                                           void *stream) {
  return block128_rows_gemm(true, dy_codes, dy_scale, w_codes, w_scale, offsets, num_experts, m, n, k, dx, dev_status,
                            stream, "grouped_gemm_dgrad_fp8_block128 launch");
}

fme_status grouped_gemm_wgrad_fp8_block128(const uint8_t *dy_codes, const float *dy_scale, const uint8_t *x_codes,
                                           const float *x_scale, int64_t positions, const int32_t *padded_offsets,
                                           int32_t num_experts, int64_t n, int64_t k, void *dw, int32_t dw_mode,
                                           int32_t *dev_status, void *stream) {
  if (n < 0 || k < 0 || positions < 0 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (dw_mode != FME_DW_BF16 && dw_mode != FME_DW_FP32 && dw_mode != FME_DW_FP32_ADD) return FME_ERR_INVALID_ARGUMENT;
  if (!block128_cols(n) || !block128_cols(k) || positions % 128 != 0 || positions > (int64_t(1) << 31) - 1)
    return FME_ERR_UNSUPPORTED_SHAPE;
  if (num_experts * ((n + 255) / 256) * ((k + 255) / 256) > (int64_t(1) << 31) - 1 ||
      num_experts * n > (int64_t(1) << 31) - 1 - 256)
    return FME_ERR_UNSUPPORTED_SHAPE;
  if (!padded_offsets || !dw) return FME_ERR_INVALID_ARGUMENT;
  if (positions > 0 && (!dy_codes || !dy_scale || !x_codes || !x_scale)) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(dy_codes) || !aligned16(dy_scale) || !aligned16(x_codes) || !aligned16(x_scale) || !aligned16(dw) ||
      !aligned16(padded_offsets))
    return FME_ERR_MISALIGNED;
  fme::LaunchBlock128 a{};
  fme_status st = current_device(&a.num_sms);
  if (st != FME_OK) return st;
  // without positions every expert is empty and the operands' maps are never used
  const void *abase = positions ? static_cast<const void *>(dy_codes) : dw;
  const void *bbase = positions ? static_cast<const void *>(x_codes) : dw;
  const int64_t extent = positions ? positions : 1;
  if ((st = encode_u8_2d(&a.map_a, abase, n, extent, n, 128)) != FME_OK) return st;
  if ((st = encode_u8_2d(&a.map_b, bbase, k, extent, k, 128)) != FME_OK) return st;
  if ((st = encode_bf16_out(&a.map_y, dw, k, static_cast<uint64_t>(num_experts) * n,
                            dw_mode == FME_DW_BF16 ? OutBox::kWideBf16 : OutBox::kWideFp32)) != FME_OK)
    return st;
  a.a_scale = dy_scale;
  a.b_scale = x_scale;
  a.offsets = padded_offsets;
  a.num_experts = num_experts;
  a.m = n;
  a.n = k;
  a.positions = positions;
  a.y = dw;
  a.out_fp32 = dw_mode != FME_DW_BF16;
  a.accumulate = dw_mode == FME_DW_FP32_ADD;
  a.status = dev_status;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_block128_wgrad(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "grouped_gemm_wgrad_fp8_block128 launch");
}

// -------------------------------------------------------------- bf16 products --
namespace {

// Columns of a bf16 operand: its rows are a multiple of 16 bytes.
bool bf16_cols(int64_t c) { return c >= 8 && c <= 65536 && c % 8 == 0; }

// 2-D bf16 matrix [rows x cols], boxes of 128 bytes x box_rows, 128-byte swizzle, zero fill out of bounds.
fme_status encode_bf16_2d(CUtensorMap *map, const void *base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {64, box_rows};
  return encode_map(" (rows)", map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// 3-D bf16 weights [experts][n][k], the same boxes, zero fill past each expert's n and k.
fme_status encode_bf16_weights(CUtensorMap *map, const void *base, uint64_t experts, uint64_t n, uint64_t k,
                               uint32_t box_rows) {
  cuuint64_t dims[3] = {k, n, experts};
  cuuint64_t strides[2] = {k * 2, n * k * 2};
  cuuint32_t box[3] = {64, box_rows, 1};
  return encode_map(" (weights)", map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// MN-major weights, 64 rows x 128 columns: with whole groups of 64 columns, one box that gives them as two of 64 columns
// one after the other ([experts][cols / 64][rows][64]); otherwise boxes of 64 columns, cut at the row's end.
fme_status encode_bf16_mn(CUtensorMap *map, bool *wide, const void *base, uint64_t experts, uint64_t rows, uint64_t cols) {
  *wide = cols % 64 == 0;
  if (!*wide) return encode_bf16_weights(map, base, experts, rows, cols, 64);
  cuuint64_t dims[4] = {64, rows, cols / 64, experts};
  cuuint64_t strides[3] = {cols * 2, 128, rows * cols * 2};
  cuuint32_t box[4] = {64, 64, 2, 1};
  return encode_map(" (columns)", map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// wgrad's operands, from 64 rows on: all windows of 64 rows of a matrix, window s its rows s .. s + 63 (from window to window
// the stride is a row's), in the same boxes.  One that starts at row 64 - c of window s holds rows s + 64 - c .. s + 63 and
// zeros behind them.
fme_status encode_bf16_windows(CUtensorMap *map, bool *wide, const void *base, uint64_t rows, uint64_t cols) {
  *wide = cols % 64 == 0;
  cuuint64_t dims[4] = {64, 64, cols / 64, rows - 63};
  cuuint64_t strides[3] = {cols * 2, 128, cols * 2};
  cuuint32_t box[4] = {64, 64, 2, 1};
  if (!*wide) {
    dims[0] = cols;
    dims[2] = rows - 63;
    strides[1] = cols * 2;
    box[2] = 1;
  }
  return encode_map(" (windows)", map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, *wide ? 4 : 3, const_cast<void *>(base), dims, strides,
                    box, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// The forward (out = n columns, contraction k) and dgrad (out = k columns, contraction n).
fme_status bf16_rows_gemm(bool dgrad, const void *a_rows, const void *w, const int32_t *offsets, int32_t num_experts,
                          int64_t m, int64_t n, int64_t k, void *y, int32_t *dev_status, void *stream,
                          const char *what) {
  if (m < 0 || n < 0 || k < 0 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (!bf16_cols(n) || !bf16_cols(k)) return FME_ERR_UNSUPPORTED_SHAPE;
  // row coordinates of the last, partly empty tiles and the number of tiles stay in 32 bits
  if (m > (int64_t(1) << 31) - 1 - 256) return FME_ERR_UNSUPPORTED_SHAPE;
  if ((m / 64 + num_experts) * (((dgrad ? k : n) + 127) / 128) > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  if (!offsets) return FME_ERR_INVALID_ARGUMENT;
  if (m == 0) return FME_OK;
  if (!a_rows || !w || !y) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(a_rows) || !aligned16(w) || !aligned16(y) || !aligned16(offsets)) return FME_ERR_MISALIGNED;
  fme::LaunchBf16 a{};
  fme_status st = current_device(&a.num_sms);
  if (st != FME_OK) return st;
  a.k = dgrad ? n : k;
  a.n = dgrad ? k : n;
  a.few_halves = dgrad ? 0 : fme::bf16_few_halves(m, n, k, num_experts, a.num_sms);
  const bool few = a.few_halves != 0;
  CUtensorMap &rows_map = few ? a.map_b : a.map_a, &w_map = few ? a.map_a : a.map_b;
  if ((st = encode_bf16_2d(&rows_map, a_rows, m, a.k, few ? 16 : 128)) != FME_OK) return st;
  st = dgrad ? encode_bf16_mn(&w_map, &a.wide_b, w, num_experts, n, k)
             : encode_bf16_weights(&w_map, w, num_experts, n, k, few ? 256 / a.few_halves : 128);
  if (st != FME_OK) return st;
  if ((st = encode_bf16_out(&a.map_y, y, a.n, m, OutBox::kWideBf16)) != FME_OK) return st;
  a.offsets = offsets;
  a.num_experts = num_experts;
  a.rows = m;
  a.m = m;
  a.y = y;
  a.status = dev_status;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = dgrad ? fme::launch_bf16_dgrad(a) : fme::launch_bf16_fwd(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, what);
}

}  // namespace

fme_status grouped_gemm_fwd_bf16(const void *x, const void *w, const int32_t *offsets, int32_t num_experts, int64_t m,
                                 int64_t n, int64_t k, void *y, int32_t *dev_status, void *stream) {
  return bf16_rows_gemm(false, x, w, offsets, num_experts, m, n, k, y, dev_status, stream,
                        "grouped_gemm_fwd_bf16 launch");
}

fme_status grouped_gemm_dgrad_bf16(const void *dy, const void *w, const int32_t *offsets, int32_t num_experts, int64_t m,
                                   int64_t n, int64_t k, void *dx, int32_t *dev_status, void *stream) {
  return bf16_rows_gemm(true, dy, w, offsets, num_experts, m, n, k, dx, dev_status, stream,
                        "grouped_gemm_dgrad_bf16 launch");
}

fme_status grouped_gemm_wgrad_bf16(const void *dy, const void *x, int64_t m, const int32_t *offsets, int32_t num_experts,
                                   int64_t n, int64_t k, void *dw, int32_t dw_mode, int32_t *dev_status, void *stream) {
  if (n < 0 || k < 0 || m < 0 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (dw_mode != FME_DW_BF16 && dw_mode != FME_DW_FP32 && dw_mode != FME_DW_FP32_ADD) return FME_ERR_INVALID_ARGUMENT;
  if (!bf16_cols(n) || !bf16_cols(k) || m > (int64_t(1) << 31) - 1 - 256) return FME_ERR_UNSUPPORTED_SHAPE;
  if (num_experts * ((n + 255) / 256) * ((k + 255) / 256) > (int64_t(1) << 31) - 1 ||
      num_experts * n > (int64_t(1) << 31) - 1 - 256)
    return FME_ERR_UNSUPPORTED_SHAPE;
  if (!offsets || !dw) return FME_ERR_INVALID_ARGUMENT;
  if (m > 0 && (!dy || !x)) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(dy) || !aligned16(x) || !aligned16(dw) || !aligned16(offsets)) return FME_ERR_MISALIGNED;
  fme::LaunchBf16 a{};
  fme_status st = current_device(&a.num_sms);
  if (st != FME_OK) return st;
  // without rows every expert is empty and the operands' maps are never used
  const void *abase = m ? dy : dw, *bbase = m ? x : dw;
  const int64_t extent = m ? m : 1;
  if ((st = encode_bf16_2d(&a.early_a, abase, extent, n, 64)) != FME_OK ||
      (st = encode_bf16_2d(&a.early_b, bbase, extent, k, 64)) != FME_OK)
    return st;
  a.map_a = a.early_a;  // with fewer rows than a window every block is an early one
  a.map_b = a.early_b;
  if (m >= 64 && ((st = encode_bf16_windows(&a.map_a, &a.wide_a, dy, m, n)) != FME_OK ||
                  (st = encode_bf16_windows(&a.map_b, &a.wide_b, x, m, k)) != FME_OK))
    return st;
  a.offsets = offsets;
  a.num_experts = num_experts;
  a.rows = m;
  a.m = n;
  a.n = k;
  a.y = dw;
  a.out_fp32 = dw_mode != FME_DW_BF16;
  a.accumulate = dw_mode == FME_DW_FP32_ADD;
  a.status = dev_status;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_bf16_wgrad(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "grouped_gemm_wgrad_bf16 launch");
}

// ----------------------------------------------- NVFP4 weights, few bf16 rows --
namespace {

// Tiled scales as [groups of 128 rows][tiles][512 bytes], boxes of 4 tiles x the 128 bytes of 8 rows of each quarter, zero
// fill past a row's last tile.
fme_status encode_scale_tiles(CUtensorMap *map, const void *base, uint64_t groups, uint64_t tiles) {
  cuuint64_t dims[3] = {512, tiles, groups};
  cuuint64_t strides[2] = {512, tiles * 512};
  cuuint32_t box[3] = {128, 4, 1};
  return encode_map(" (scale tiles)", map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

fme_status gemv_nvfp4(bool swiglu, const void *x, int64_t x_rows, const int32_t *src_row, int32_t top_k,
                      const uint8_t *w_codes, const uint8_t *w_sf, const float *w_scale, const int32_t *offsets,
                      int32_t num_experts, int64_t m, int64_t n, int64_t k, void *y, int32_t *dev_status, void *stream,
                      const char *what) {
  if (m < 0 || n < 0 || k < 0 || x_rows < 0 || check_groups(num_experts) != FME_OK) return FME_ERR_INVALID_ARGUMENT;
  if (top_k < 1 || top_k > 64) return FME_ERR_INVALID_ARGUMENT;
  if (x_rows > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  if (src_row ? m != x_rows * top_k : m != x_rows || top_k != 1) return FME_ERR_INVALID_ARGUMENT;
  if (k % 64 != 0 || k < 64 || k > 8192 || n < 1 || n > 65536 || (swiglu && n % 256 != 0)) return FME_ERR_UNSUPPORTED_SHAPE;
  // the number of units, of 4 rows and 32 weight rows at least, stays in 32 bits
  if (m > (int64_t(1) << 31) - 1 - 256 || (m / 4 + num_experts) * ((n + 254) / 128) * 4 > (int64_t(1) << 31) - 1)
    return FME_ERR_UNSUPPORTED_SHAPE;
  if (!offsets) return FME_ERR_INVALID_ARGUMENT;
  if (m == 0) return FME_OK;
  if (!x || !w_codes || !w_sf || !w_scale || !y) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(src_row) || !aligned16(w_codes) || !aligned16(w_sf) || !aligned16(w_scale) ||
      !aligned16(y) || !aligned16(offsets))
    return FME_ERR_MISALIGNED;
  fme::LaunchGemv a{};
  fme_status st = current_device(&a.num_sms);
  if (st != FME_OK) return st;
  a.x = x;
  a.x_rows = x_rows;
  a.src_row = src_row;
  a.top_k = top_k;
  const uint64_t w_rows = static_cast<uint64_t>(num_experts) * n;
  if ((st = encode_u8_2d(&a.map_codes, w_codes, k / 2, w_rows, k / 2, 8)) != FME_OK) return st;
  if ((st = encode_scale_tiles(&a.map_sf, w_sf, (w_rows + 127) / 128, k / 64)) != FME_OK) return st;
  a.scale = w_scale;
  a.offsets = offsets;
  a.num_experts = num_experts;
  a.m = m;
  a.n = n;
  a.k = k;
  a.swiglu = swiglu;
  a.y = y;
  a.status = dev_status;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_gemv_nvfp4(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, what);
}

}  // namespace

fme_status grouped_gemv_nvfp4(const void *x, int64_t x_rows, const int32_t *src_row, int32_t top_k,
                              const uint8_t *w_codes, const uint8_t *w_sf, const float *w_scale, const int32_t *offsets,
                              int32_t num_experts, int64_t m, int64_t n, int64_t k, void *y, int32_t *dev_status,
                              void *stream) {
  return gemv_nvfp4(false, x, x_rows, src_row, top_k, w_codes, w_sf, w_scale, offsets, num_experts, m, n, k, y, dev_status,
                    stream, "grouped_gemv_nvfp4 launch");
}

fme_status grouped_gemv_nvfp4_swiglu(const void *x, int64_t x_rows, const int32_t *src_row, int32_t top_k,
                                     const uint8_t *w_codes, const uint8_t *w_sf, const float *w_scale,
                                     const int32_t *offsets, int32_t num_experts, int64_t m, int64_t n, int64_t k, void *h,
                                     int32_t *dev_status, void *stream) {
  return gemv_nvfp4(true, x, x_rows, src_row, top_k, w_codes, w_sf, w_scale, offsets, num_experts, m, n, k, h, dev_status,
                    stream, "grouped_gemv_nvfp4_swiglu launch");
}

// ------------------------------------------------- SwiGLU and grouping in bf16 --
namespace {

fme_status swiglu_bf16(const void *gate_up, const void *dh, bool backward, int64_t rows, int64_t inter, void *out,
                       void *stream, const char *what) {
  if (rows < 0 || inter < 0) return FME_ERR_INVALID_ARGUMENT;
  if (inter < 8 || inter > 65536 || inter % 8 != 0 || rows > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  if (rows * (inter / 8) / 1024 > (int64_t(1) << 31) - 2) return FME_ERR_UNSUPPORTED_SHAPE;  // CTAs
  if (rows == 0) return FME_OK;
  if (!gate_up || !out || (backward && !dh)) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(gate_up) || !aligned16(dh) || !aligned16(out)) return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  cudaError_t err = fme::launch_swiglu({gate_up, dh, rows, inter, out, static_cast<cudaStream_t>(stream)});
  return err == cudaSuccess ? FME_OK : cuda_fail(err, what);
}

}  // namespace

fme_status swiglu(const void *gate_up, int64_t rows, int64_t inter, void *h, void *stream) {
  return swiglu_bf16(gate_up, nullptr, false, rows, inter, h, stream, "swiglu launch");
}

fme_status swiglu_backward(const void *gate_up, const void *dh, int64_t rows, int64_t inter, void *d_gate_up,
                           void *stream) {
  return swiglu_bf16(gate_up, dh, true, rows, inter, d_gate_up, stream, "swiglu_backward launch");
}

fme_status moe_permute(const void *x, int64_t tokens, int64_t n, const int32_t *src_row, int32_t top_k, void *out,
                       int32_t *dev_status, void *stream) {
  if (tokens < 0 || n < 0 || top_k < 1 || top_k > 64) return FME_ERR_INVALID_ARGUMENT;
  if (n < 8 || n > 65536 || n % 8 != 0 || tokens > ((int64_t(1) << 31) - 1) / top_k) return FME_ERR_UNSUPPORTED_SHAPE;
  if (tokens * top_k * (n / 8) / 1024 > (int64_t(1) << 31) - 1 - 64) return FME_ERR_UNSUPPORTED_SHAPE;  // CTAs
  if (tokens == 0) return FME_OK;
  if (!x || !src_row || !out) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(src_row) || !aligned16(out)) return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  cudaError_t err =
      fme::launch_permute({x, src_row, tokens, top_k, n, out, dev_status, static_cast<cudaStream_t>(stream)});
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "moe_permute launch");
}

// ------------------------------------------------------------------ router --
namespace {

// Tokens are summed in equal chunks, a CTA each: two CTAs for every SM at most, 16 tokens (one a
// warp) at least.  A function of the sizes alone, so that the workspace and the order of the sums do
// not depend on the device.
int64_t balance_chunk(int64_t tokens) {
  const int64_t c = (tokens + 303) / 304;
  return c < 16 ? 16 : c;
}

int64_t round16(int64_t b) { return (b + 15) / 16 * 16; }

struct BalanceWorkspace {
  int64_t sums, counts, tokens, term, flags, bytes;
};
BalanceWorkspace balance_workspace(int64_t tokens, int64_t num_seqs, int32_t num_experts) {
  const int64_t chunk = balance_chunk(tokens);
  const int64_t slots = (tokens + chunk - 1) / chunk + num_seqs;
  BalanceWorkspace w;
  w.sums = 0;
  w.counts = w.sums + round16(slots * num_experts * 4);
  w.tokens = w.counts + round16(slots * num_experts * 4);
  w.term = w.tokens + round16(slots * 4);
  w.flags = w.term + round16(num_seqs * ((num_experts + 31) / 32) * 4);
  w.bytes = w.flags + 16;
  return w;
}

bool router_dtype(int32_t d) { return d == FME_BF16 || d == FME_FP32; }
bool router_score(int32_t s) { return s == FME_SCORE_SOFTMAX || s == FME_SCORE_SIGMOID; }

// Sizes common to the router's calls.
fme_status check_router(int64_t tokens, int32_t num_experts, int32_t top_k, int32_t dtype, int32_t score) {
  if (tokens < 0 || num_experts < 1 || top_k < 1 || top_k > num_experts) return FME_ERR_INVALID_ARGUMENT;
  if (!router_dtype(dtype) || !router_score(score)) return FME_ERR_INVALID_ARGUMENT;
  if (num_experts > FME_MAX_GROUPS || top_k > 32 || tokens > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  return FME_OK;
}

}  // namespace

int64_t fme_balance_workspace_bytes(int64_t tokens, int64_t num_seqs, int32_t num_experts) {
  if (tokens < 0 || num_seqs < 1 || num_experts < 1) return 0;
  return balance_workspace(tokens, num_seqs, num_experts).bytes;
}

fme_status moe_gate(const void *logits, int32_t dtype, int64_t tokens, int32_t num_experts, int32_t top_k, int32_t score,
                    int32_t normalize, float scale, const float *bias, int32_t *ids, float *weights, void *stream) {
  fme_status st = check_router(tokens, num_experts, top_k, dtype, score);
  if (st != FME_OK) return st;
  if (tokens == 0) return FME_OK;
  if (!logits || !ids || !weights) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(logits) || !aligned16(bias) || !aligned16(ids) || !aligned16(weights)) return FME_ERR_MISALIGNED;
  int sms = 0;
  if ((st = current_device(&sms)) != FME_OK) return st;
  fme::LaunchGate a{};
  a.logits = logits;
  a.bf16 = dtype == FME_BF16;
  a.tokens = tokens;
  a.num_experts = num_experts;
  a.top_k = top_k;
  a.softmax = score == FME_SCORE_SOFTMAX;
  a.normalize = normalize != 0;
  a.scale = scale;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_gate(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "moe_gate launch");
}

fme_status moe_gate_backward(const void *logits, int32_t dtype, const int32_t *ids, const float *d_weights,
                             int64_t tokens, int32_t num_experts, int32_t top_k, int32_t score, int32_t normalize,
                             float scale, void *d_logits, int32_t *dev_status, void *stream) {
  fme_status st = check_router(tokens, num_experts, top_k, dtype, score);
  if (st != FME_OK) return st;
  if (tokens == 0) return FME_OK;
  if (!logits || !ids || !d_weights || !d_logits) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(logits) || !aligned16(ids) || !aligned16(d_weights) || !aligned16(d_logits)) return FME_ERR_MISALIGNED;
  int sms = 0;
  if ((st = current_device(&sms)) != FME_OK) return st;
  fme::LaunchGate a{};
  a.logits = logits;
  a.bf16 = dtype == FME_BF16;
  a.tokens = tokens;
  a.num_experts = num_experts;
  a.top_k = top_k;
  a.softmax = score == FME_SCORE_SOFTMAX;
  a.normalize = normalize != 0;
  a.scale = scale;
  a.ids = const_cast<int32_t *>(ids);
  a.d_weights = d_weights;
  a.d_logits = d_logits;
  a.status = dev_status;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_gate_backward(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "moe_gate_backward launch");
}

fme_status moe_balance_loss(const void *logits, int32_t dtype, const int32_t *ids, int64_t tokens, int32_t num_experts,
                            int32_t top_k, int32_t score, float alpha, const int32_t *seq_offsets, int64_t num_seqs,
                            const uint8_t *token_mask, float *loss, int32_t *counts, int32_t *seq_tokens,
                            void *workspace, int64_t workspace_bytes, int32_t *dev_status, void *stream) {
  fme_status st = check_router(tokens, num_experts, top_k, dtype, score);
  if (st != FME_OK) return st;
  if (num_seqs < 1 || (!seq_offsets && num_seqs != 1)) return FME_ERR_INVALID_ARGUMENT;
  if (num_seqs > (int64_t(1) << 24)) return FME_ERR_UNSUPPORTED_SHAPE;  // CTAs: times ceil(1024 / 32)
  if (!loss || !counts || !seq_tokens || !workspace || (tokens > 0 && (!logits || !ids))) return FME_ERR_INVALID_ARGUMENT;
  const BalanceWorkspace w = balance_workspace(tokens, num_seqs, num_experts);
  if (workspace_bytes < w.bytes) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(logits) || !aligned16(ids) || !aligned16(seq_offsets) || !aligned16(token_mask) || !aligned16(loss) ||
      !aligned16(counts) || !aligned16(seq_tokens) || !aligned16(workspace))
    return FME_ERR_MISALIGNED;
  int sms = 0;
  if ((st = current_device(&sms)) != FME_OK) return st;
  fme::LaunchBalance a{};
  a.logits = logits;
  a.bf16 = dtype == FME_BF16;
  a.tokens = tokens;
  a.num_experts = num_experts;
  a.top_k = top_k;
  a.softmax = score == FME_SCORE_SOFTMAX;
  a.alpha = alpha;
  a.ids = ids;
  a.seq_offsets = seq_offsets;
  a.num_seqs = num_seqs;
  a.token_mask = token_mask;
  a.loss = loss;
  a.counts = counts;
  a.seq_tokens = seq_tokens;
  a.chunk = balance_chunk(tokens);
  uint8_t *base = static_cast<uint8_t *>(workspace);
  a.part_sum = reinterpret_cast<float *>(base + w.sums);
  a.part_count = reinterpret_cast<int32_t *>(base + w.counts);
  a.part_tokens = reinterpret_cast<int32_t *>(base + w.tokens);
  a.term = reinterpret_cast<float *>(base + w.term);
  a.flags = reinterpret_cast<int32_t *>(base + w.flags);
  a.status = dev_status;
  a.num_sms = sms;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_balance_loss(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "moe_balance_loss launch");
}

fme_status moe_balance_loss_backward(const void *logits, int32_t dtype, const int32_t *counts, const int32_t *seq_tokens,
                                     const float *d_loss, int64_t tokens, int32_t num_experts, int32_t top_k,
                                     int32_t score, float alpha, const int32_t *seq_offsets, int64_t num_seqs,
                                     const uint8_t *token_mask, void *d_logits, int32_t accumulate, void *stream) {
  fme_status st = check_router(tokens, num_experts, top_k, dtype, score);
  if (st != FME_OK) return st;
  if (num_seqs < 1 || (!seq_offsets && num_seqs != 1)) return FME_ERR_INVALID_ARGUMENT;
  if (num_seqs > (int64_t(1) << 24)) return FME_ERR_UNSUPPORTED_SHAPE;
  if (tokens == 0) return FME_OK;
  if (!logits || !counts || !seq_tokens || !d_loss || !d_logits) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(logits) || !aligned16(counts) || !aligned16(seq_tokens) || !aligned16(d_loss) ||
      !aligned16(seq_offsets) || !aligned16(token_mask) || !aligned16(d_logits))
    return FME_ERR_MISALIGNED;
  int sms = 0;
  if ((st = current_device(&sms)) != FME_OK) return st;
  fme::LaunchBalance a{};
  a.logits = logits;
  a.bf16 = dtype == FME_BF16;
  a.tokens = tokens;
  a.num_experts = num_experts;
  a.top_k = top_k;
  a.softmax = score == FME_SCORE_SOFTMAX;
  a.alpha = alpha;
  a.seq_offsets = seq_offsets;
  a.num_seqs = num_seqs;
  a.token_mask = token_mask;
  a.counts = const_cast<int32_t *>(counts);
  a.seq_tokens = const_cast<int32_t *>(seq_tokens);
  a.d_loss = d_loss;
  a.d_logits = d_logits;
  a.accumulate = accumulate != 0;
  a.num_sms = sms;
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t err = fme::launch_balance_backward(a);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "moe_balance_loss_backward launch");
}

fme_status moe_combine_backward(const void *d_out, const void *y, int64_t rows_y, const int32_t *row_of,
                                const float *weights, int64_t tokens, int32_t top_k, int64_t n, void *d_y,
                                float *d_weights, int32_t *dev_status, void *stream) {
  if (tokens < 0 || rows_y < 0 || top_k < 1 || top_k > 64 || n < 0) return FME_ERR_INVALID_ARGUMENT;
  if (n % 8 != 0 || n == 0 || n > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  if (tokens > ((int64_t(1) << 31) - 1) / top_k || rows_y > (int64_t(1) << 31) - 1) return FME_ERR_UNSUPPORTED_SHAPE;
  if (tokens == 0) return FME_OK;
  if (!d_out || !row_of || !weights || !d_weights || (rows_y > 0 && (!y || !d_y))) return FME_ERR_INVALID_ARGUMENT;
  if (!aligned16(d_out) || !aligned16(y) || !aligned16(row_of) || !aligned16(weights) || !aligned16(d_y) ||
      !aligned16(d_weights))
    return FME_ERR_MISALIGNED;
  int sms = 0;
  fme_status st = current_device(&sms);
  if (st != FME_OK) return st;
  fme::LaunchCombineBackward c{d_out, y, row_of, weights, tokens, top_k, n, rows_y, d_y, d_weights, dev_status,
                               static_cast<cudaStream_t>(stream)};
  cudaError_t err = fme::launch_combine_backward(c);
  return err == cudaSuccess ? FME_OK : cuda_fail(err, "moe_combine_backward launch");
}

}  // extern "C"
