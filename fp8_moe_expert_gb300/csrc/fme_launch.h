// fme_launch.h -- host-side launch descriptions passed from the C ABI layer
// (api.cu, which validates arguments) to the kernel launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
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

// bf16 grouped GEMMs (gemm_bf16.cu).
struct LaunchBf16 {
  CUtensorMap map_a, map_b;      // operands, 128-byte swizzle (wgrad: all windows of 64 rows; not with fewer rows)
  CUtensorMap early_a, early_b;  // wgrad: the operands in boxes of 64 rows x 64 columns
  CUtensorMap map_y;             // output (not wgrad's), boxes of 32 rows x 128 bytes, 128-byte swizzle
  const int32_t *offsets;  // rows of each expert
  int32_t num_experts;
  int64_t rows;     // rows of all experts
  int64_t m, n, k;  // output rows (wgrad: of one expert) and columns; contraction (not wgrad)
  void *y;
  bool out_fp32, accumulate;  // wgrad
  int few_halves;             // forward: bf16_few_halves
  bool wide_a, wide_b;        // MN-major operands: the map gives 128 columns as two of 64 in one box
  int32_t *status;
  int num_sms;
  int stages;  // operand ring depth, set by the launcher
  cudaStream_t stream;
};
// At most so many tiles of 64 tokens: each expert with a row has one, and 64 more rows make one more.
inline int64_t bf16_few_tiles(int64_t m, int32_t num_experts) {
  const int64_t experts = std::min<int64_t>(num_experts, m);
  return experts + (m - experts) / 64;
}
// The forward takes its few-rows form (map_a = weights, map_b = tokens in 16-row
// boxes) up to this many rows: there it reads the weights once, past it the token tiles of 64 read them again and again.  It is
// also taken while every item has an SM to itself.  Measured, us (few rows / pairs), even loads: 32 experts of 4096 x 7168, 1024
// rows 270 / 293, 2048 rows 277 / 315, 3000 rows 370 / 324; one expert, 16 rows 23 / 36, 256 rows 28 / 36, 384 rows 52 / 37; 8 experts of
// 1048 x 1400, 400 rows 11 / 14, 1400 rows 18 / 15; 4 experts of 7168 x 2048, 256 rows 25 / 29, 768 rows 42 / 31.  Where the pairs take
// over depends on the loads, which the host does not know, more than on n and k.  Over eight shapes (n 512 to 9728, k 1024 to
// 7168) and 1 to 32 experts, where the items are more than the SMs: with even loads the form for few rows is ahead in all 26
// up to 64 rows an expert (there by 4 to 15%), the pairs in 25 from 80 on (by up to a third); with Zipf loads it is ahead in
// all 17 at 16 rows an expert, in 17 of 20 at 32, 8 at 40, 5 at 48 and 3 at 64 (the pairs by up to 27%).  The border is between.
// Returns 0 where not; otherwise the blocks of 64 of k in a stage, 2, 4 or 8 for items of 128, 64 or 32 rows of W (the boxes of
// map_a): the smaller ones while each has an SM to itself.  Items of 32 rows take more than half of the SMs only with a longer k:
// the others are left to the kernel behind, which sets itself up there (1 us).  Measured, us (8 / 4 / 2 blocks): 4096 x 7168, one
// expert, 1 or 16 rows 16.6 / 18.7 / 23.0, 32 rows - / 19.4 / 23.6; of seven shapes of 112 to 152 items of 32, with k 1536 and less
// items of 64 are ahead by up to 10% (3584 x 512: 4.3 / 3.8), with 2048 and 2560 they differ by 4% at most, with 3584 and more items of
// 32 are ahead in all (3584 x 4096: 11.0 / 11.9).  Of 13 shapes of 112 to 152 items of 64 they are ahead of 128 rows, or within 2%, for
// every k from 512 to 7168 (7168 x 2048: 8.9 / 9.5; x 1024: 6.4 / 6.4).
inline int bf16_few_halves(int64_t m, int64_t n, int64_t k, int32_t num_experts, int num_sms) {
  const int64_t tiles = bf16_few_tiles(m, num_experts);
  auto alone = [&](int64_t rows, int sms) { return tiles * ((n + rows - 1) / rows) <= sms; };
  if (m > 16 + 48 * static_cast<int64_t>(num_experts) && !alone(128, num_sms)) return 0;
  if (m <= 16 && alone(32, k >= 2560 ? num_sms : num_sms / 2)) return 8;
  return m <= 32 && alone(64, num_sms) ? 4 : 2;
}
cudaError_t launch_bf16_fwd(const LaunchBf16 &a);
cudaError_t launch_bf16_dgrad(const LaunchBf16 &a);
cudaError_t launch_bf16_wgrad(const LaunchBf16 &a);

// Few bf16 rows times NVFP4 weights (gemv_nvfp4.cu).
struct LaunchGemv {
  CUtensorMap map_codes;  // [weight rows x k / 2], boxes of 8 rows x 128 bytes, 128-byte swizzle
  CUtensorMap map_sf;     // [groups of 128 rows][k / 64 tiles][512 bytes], boxes of 4 tiles x 128 bytes
  const void *x;
  int64_t x_rows;
  const int32_t *src_row;  // or NULL
  int32_t top_k;
  const float *scale;
  const int32_t *offsets;
  int32_t num_experts;
  int64_t m, n, k;
  bool swiglu;
  void *y;
  int32_t *status;
  int num_sms;
  int32_t tile_rows;      // set by the launcher: rows of x at a time,
  uint32_t shared_bytes;  // and what there is of shared memory
  cudaStream_t stream;
};
// Rows of x taken at a time, at most: eight with 7168 of k are half of an SM's shared memory.
constexpr int kGemvRows = 8;
inline int32_t gemv_tile_rows(int64_t k) { return k <= 7168 ? kGemvRows : kGemvRows / 2; }
// An upper bound of a call's units: every expert with a row has a tile, and each further one takes as many rows as a tile.
inline int64_t gemv_units(bool swiglu, int64_t m, int64_t n, int64_t k, int32_t num_experts) {
  const int64_t per = swiglu ? n / 256 * 8 : (n % 128 == 0 ? n / 128 : (n + 254) / 128) * 4;
  const int64_t experts = std::min<int64_t>(num_experts, m);
  return (experts + (m - experts) / gemv_tile_rows(k)) * per;
}
// How many warps share a unit: eight while the SMs have few, four from two units an SM on; two where the chunks of 256 k would
// leave some of four without work and not of two.  Measured, us with 8 / 4 / 2 warps, experts with a row each: gate/up of 4096 x 7168
// with SwiGLU, one (0.8 units an SM) 9.1 / 11.2 / 19.3, two (1.7) 11.6 / 13.2 / 19.7, three (2.5) 15.8 / 15.1 / 20.9, eight (7)
// 31.6 / 30.0 / 31.0, 32 (27) 98 / 91 / 97; down projection of 7168 x 2048, one (1.5) 6.7 / 7.1 / 8.9, eight (12) 19.6 / 18.2 / 19.0,
// 32 (47) 59 / 52 / 50, with 128 rows in all 63 / 57 / 59; 4096 x 1536, four (3.4) 9.1 / 8.9 / 8.6, 32 (27) 35 / 33 / 29; 4096 x
// 2304, four 10.8 / 10.2 / 10.5, 32 50 / 44 / 40; 2048 x 512, eight (3.4) 7.5 / 6.7 / 6.2.  Over 476 shapes (k 256 to 7168, 4 and 16
// experts with a row each, 1 to 16 units an SM, with and without SwiGLU) the choice is 1% behind the fastest of the three on the
// average, and 15% at most (13 chunks, five units an SM, where two warps would be it).  A rule of its own for five and six chunks
// is not there: with two to five units an SM eight warps are behind four in all 28 of those shapes, though 74 rows of 8 experts of
// 1000 x 1344 take 11.2 / 11.8 / 13.8.
inline int gemv_share(int64_t units, int64_t k, int num_sms) {
  if (units < 2 * num_sms) return 8;
  const int64_t chunks = (k + 255) / 256;
  const bool uneven = chunks <= 10 && (chunks % 4 == 1 || chunks % 4 == 2);
  return uneven && (units >= 5 * num_sms || chunks <= 2) ? 2 : 4;
}
cudaError_t launch_gemv_nvfp4(const LaunchGemv &a);

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

struct LaunchPermute {
  const void *x;
  const int32_t *src_row;
  int64_t tokens;
  int32_t top_k;
  int64_t n;
  void *out;
  int32_t *status;
  cudaStream_t stream;
};
cudaError_t launch_permute(const LaunchPermute &c);

// SwiGLU in bf16 (activation.cu): the backward with dh.
struct LaunchSwiglu {
  const void *gate_up, *dh;
  int64_t rows, inter;
  void *out;
  cudaStream_t stream;
};
cudaError_t launch_swiglu(const LaunchSwiglu &a);

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
