// fme_launch.h -- host-side launch descriptions passed from the C ABI layer
// (api.cu, which validates arguments) to the kernel launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace fme {

// Lets a kernel have as much dynamic shared memory as a block can get on the current device; `done` is the
// kernel's own (of internal linkage: a process may hold two builds), a bit for each device.  Once and never lowered:
// the limit belongs to the function, and set to each launch's own size it could be lowered by another host
// thread's call before the launch that needed it.
inline cudaError_t allow_shared(const void *kernel, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = uint64_t(1) << (dev & 63);  // current_device() admits 64
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  int most = 0;
  cudaFuncAttributes f{};
  if ((err = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess ||
      (err = cudaFuncGetAttributes(&f, kernel)) != cudaSuccess ||
      (err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  most - static_cast<int>(f.sharedSizeBytes))) != cudaSuccess)
    return err;
  done.fetch_or(bit, std::memory_order_release);
  return cudaSuccess;
}

struct LaunchNvfp4 {
  const void *x;
  int64_t rows, k;
  const int32_t *offsets;
  int32_t num_groups;
  uint8_t *codes, *sf;
  float *row_scale;
  int32_t *status;
  int num_sms;
  cudaStream_t stream;
  bool swiglu = false;         // x is a gate/up output [rows x 2k]; quantize silu(gate) * up
  void *h_out = nullptr;       // swiglu: the bf16 activation [rows x k], or NULL
  const int32_t *gather = nullptr;  // row r reads input row gather[r] / gather_div (permuted tokens)
  int32_t gather_div = 1;
  int64_t gather_limit = 0;         // input rows; gathered rows outside [0, limit) are reported
  const float *tensor_amax = nullptr;  // standard NVFP4: every row scaled by this amax (device)
};

struct LaunchRoute {
  const int32_t *ids;
  int64_t tokens;
  int32_t top_k, num_experts;
  int32_t *offsets, *row_of, *src_row;
  int32_t *ws;  // [chunks x num_experts]
  int32_t *status;
  cudaStream_t stream;
};

struct LaunchCombine {
  const void *y;
  const int32_t *row_of;
  const float *weights;
  int64_t tokens;
  int32_t top_k;
  int64_t n, rows_y;
  void *out;
  int32_t *status;
  int num_sms;
  cudaStream_t stream;
};

struct LaunchMxfp8 {
  const void *x;
  int64_t rows, cols;
  const int32_t *offsets;
  int32_t num_groups;
  uint8_t *codes, *sf;
  int32_t *padded_offsets;  // column-wise only
  int64_t ld;               // column-wise only
  int32_t *status;
  int num_sms;
  cudaStream_t stream;
  // Row-wise only: row r reads source row gather[r] / gather_div, which must lie
  // in [0, gather_limit).
  const int32_t *gather = nullptr;
  int32_t gather_div = 1;
  int64_t gather_limit = 0;
  // SwiGLU backward (launch_swiglu_bwd_mxfp8): x = gate/up [rows x cols], dh
  // [rows x cols/2], optional bf16 d(gate/up) out [rows x cols].
  const void *dh = nullptr;
  void *d_out = nullptr;
  bool ceil_scale = false;  // row-wise / column-wise only: X = 2^ceil(log2(amax / 448))
};

// kFwdNvfp4Swiglu: the NVFP4 forward of the gate/up projection with h = silu(gate) * up
// formed in the epilogue (output [rows x n / 2]).
enum class GemmKind { kFwdNvfp4 = 0, kDgradMxfp8 = 1, kWgradMxfp8 = 2, kFwdMxfp8 = 3, kFwdNvfp4Swiglu = 4 };
__host__ __device__ constexpr bool is_fwd_nvfp4(GemmKind k) {
  return k == GemmKind::kFwdNvfp4 || k == GemmKind::kFwdNvfp4Swiglu;
}

struct LaunchGemm {
  GemmKind kind;
  CUtensorMap map_a, map_b;      // operand codes, uint8, 128-byte swizzle
  CUtensorMap map_sfa, map_sfb;  // tiled scales viewed as [128-row blocks x 8-byte words]
  CUtensorMap map_y;             // the bf16 output [rows x n], 32 x 32 boxes, 64-byte swizzle (not the fp32 accumulate)
  const float *a_scale, *b_scale;  // forward only
  const int32_t *offsets;          // row offsets (fwd, dgrad) or padded offsets (wgrad)
  int32_t num_experts;
  int64_t m, n, k;          // GEMM sizes; k unused for wgrad (per-expert)
  int64_t lda, ldb;         // wgrad: position extents of A and B; dgrad: ldb
  void *y;
  int32_t *status;
  int num_sms;
  int stages;  // operand ring depth, set by launch_grouped_gemm
  cudaStream_t stream;
  bool accumulate = false;  // wgrad only: y is fp32 and receives y += result
};

// FP8 block-128 quantizers (quant_block128.cu).
struct LaunchFp8Quant {
  const void *x;
  int64_t rows, cols;       // weights: rows of one expert
  const int32_t *offsets;   // column-wise
  int32_t num_groups;       // column-wise: groups; weights: experts
  uint8_t *codes;
  float *scale;
  int32_t *padded_offsets;  // column-wise
  int64_t ld;               // column-wise: padded positions
  uint8_t *row_codes;       // column-wise: also row-wise (or NULL)
  float *row_scale;
  const int32_t *gather;    // row-wise: row r reads row gather[r] / gather_div of gather_limit (or NULL)
  int32_t gather_div;
  int64_t gather_limit;
  int32_t *status;
  int num_sms;
  cudaStream_t stream;
};
cudaError_t launch_fp8_block128_rows(const LaunchFp8Quant &a);
cudaError_t launch_fp8_block128_cols(const LaunchFp8Quant &a);
cudaError_t launch_fp8_block128_weights(const LaunchFp8Quant &a);

// FP8 block-128 grouped GEMMs (gemm_block128.cu).
struct LaunchBlock128 {
  CUtensorMap map_a, map_b;  // codes, 128 x 128-byte boxes, 128-byte swizzle (map_b 3-D [experts][n][k] but for wgrad)
  CUtensorMap map_y;         // output, boxes of 32 rows x 128 bytes, 128-byte swizzle
  const float *a_scale, *b_scale;
  const int32_t *offsets;  // rows (forward, dgrad) or padded positions (wgrad) of each expert
  int32_t num_experts;
  int64_t m, n, k;    // output rows (wgrad: of one expert) and columns; contraction (not wgrad)
  int64_t positions;  // wgrad: padded positions of the operands
  void *y;
  bool out_fp32, accumulate;  // wgrad
  int32_t *status;
  int num_sms;
  cudaStream_t stream;
};
// The forward takes its few-rows form (map_a = weights in 128-row boxes, map_b = tokens in 16-row
// boxes) up to this many rows: there it reads the weights once at the memory's rate, past it the
// token tiles of 64 read them again and again.  Measured, n = 4096, k = 7168, us (few rows / pairs):
// 32 experts, 8 rows 41 / 63, 128 rows 139 / 193, 1024 rows 168 / 203, 2048 rows 231 / 206;
// one expert, 1 row 18 / 30, 256 rows 26 / 30, 512 rows 47 / 31; n = 1040, k = 1392, 8 experts, 400 rows
// 9.7 / 11.8.
inline bool block128_few_rows(int64_t m, int32_t num_experts) {
  return m <= 256 + 32 * static_cast<int64_t>(num_experts);
}
cudaError_t launch_block128_fwd(const LaunchBlock128 &a);
cudaError_t launch_block128_dgrad(const LaunchBlock128 &a);
cudaError_t launch_block128_wgrad(const LaunchBlock128 &a);

// The router (gate.cu).
struct LaunchGate {
  const void *logits;  // [tokens x num_experts], bf16 or fp32
  bool bf16;
  int64_t tokens;
  int32_t num_experts, top_k;
  bool softmax, normalize;
  float scale;
  const float *bias;  // or NULL
  int32_t *ids;       // read by the gradient
  float *weights;
  const float *d_weights;
  void *d_logits;
  int32_t *status;
  cudaStream_t stream;
};
struct LaunchBalance {
  const void *logits;
  bool bf16;
  int64_t tokens;
  int32_t num_experts, top_k;
  bool softmax;
  float alpha;
  const int32_t *ids;
  const int32_t *seq_offsets;  // [num_seqs + 1] or NULL
  int64_t num_seqs;
  const uint8_t *token_mask;  // or NULL
  float *loss;
  int32_t *counts, *seq_tokens;
  // workspace
  int64_t chunk;  // tokens a CTA
  float *part_sum, *term;
  int32_t *part_count, *part_tokens, *flags;
  // gradient
  const float *d_loss;
  void *d_logits;
  bool accumulate;
  int32_t *status;
  int num_sms;
  cudaStream_t stream;
};
cudaError_t launch_gate(const LaunchGate &a);
cudaError_t launch_gate_backward(const LaunchGate &a);
cudaError_t launch_balance_loss(const LaunchBalance &a);
cudaError_t launch_balance_backward(const LaunchBalance &a);

struct LaunchCombineBackward {
  const void *d_out, *y;
  const int32_t *row_of;
  const float *weights;
  int64_t tokens;
  int32_t top_k;
  int64_t n, rows_y;
  void *d_y;
  float *d_weights;
  int32_t *status;
  cudaStream_t stream;
};
cudaError_t launch_combine_backward(const LaunchCombineBackward &c);

cudaError_t launch_quantize_nvfp4(const LaunchNvfp4 &a);
// Standard NVFP4 (one FP32 scale for the whole tensor): zero *tensor_amax, reduce
// max |x| into it, then quantize every row with it in place of the row's amax.
cudaError_t launch_quantize_nvfp4_pertensor(const LaunchNvfp4 &a, float *tensor_amax);
cudaError_t launch_quantize_mxfp8_rows(const LaunchMxfp8 &a);
cudaError_t launch_quantize_mxfp8_cols(const LaunchMxfp8 &a);
cudaError_t launch_quantize_mxfp8_rowcol(const LaunchMxfp8 &a, uint8_t *row_codes, uint8_t *row_sf);
// Fused SwiGLU backward + row-wise and column-wise MXFP8 of d(gate/up); a.codes /
// a.sf are the column-wise outputs (as launch_quantize_mxfp8_rowcol).
cudaError_t launch_swiglu_bwd_mxfp8(const LaunchMxfp8 &a, uint8_t *row_codes, uint8_t *row_sf);
cudaError_t launch_grouped_gemm(const LaunchGemm &a);
cudaError_t launch_route(const LaunchRoute &r);
// launch_route with the module's static device counters as the workspace (r.ws
// is ignored); needs chunks * num_experts <= kRouteStaticWords.
constexpr int64_t kRouteStaticWords = int64_t(1) << 20;
cudaError_t launch_route_static(LaunchRoute r);
cudaError_t launch_combine(const LaunchCombine &c);
constexpr int64_t kRouteChunkHost = 1024;  // assignments per routing chunk (route.cu)

}  // namespace fme
