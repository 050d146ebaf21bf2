// gemv_nvfp4.cu -- products of few bf16 rows with NVFP4 expert weights, for decode steps.
//
//   y[t, n] = S[e, n] sum_k x[t, k] c[e, n, k] sf[e, n, k / 16]      (t a row of expert e)
//
// from the codes c (E2M1), block scales sf (E4M3) and row scales S (fp32) of quantize_nvfp4_pertoken, the same weights
// as grouped_gemm_fwd_nvfp4's, with activations that stay bf16 ("Composer 2 Technical Report", section 6.1, the
// NVFP4 variant of the forward; for a few rows the time is that of reading the weights, and quantizing the rows would save
// nothing).  With SwiGLU the gate and the matching up rows are taken together and h = silu(g) u leaves.
//
// An E2M1 code times an E4M3 scale has at most six significant bits and lies in 2^-10 .. 2688, so it is a bf16 value
// exactly: the weights are turned into bf16 fragments in registers and multiplied by mma.sync (m16n8k16, fp32 sums).  A
// warp-wide MMA fits here where tcgen05 does not: its A operand may come from registers, and with at most 8 rows (its
// N) the tensor work is a tenth of the decoding's time.
//
// Decoding 8 codes of a word: two of them lie 16 bits apart, one in each half of the word.  A masked pair times
// (2^12 + 2^6) puts a code's sign into bit 15 and its exponent and mantissa into bits 8 .. 6 of each half: as bf16 that is
// the code's value times 2^-126 (its subnormal 0.5 a bf16 subnormal).  Times sf 2^118, one packed product, it is c sf 2^-8, exact.  The 2^8 is put
// back with the row scale.  13 integer operations and 4 products for 8 weights.
//
// Any order of k will do as long as both operands follow it.  Lane (g, t) = (lane / 4, lane % 4) of a warp takes 32
// consecutive k of a chunk of 128 for rows g, g + 32, g + 64 and g + 96 of a group of 128 weight rows: one
// 16-byte load a row for the codes and one for the scales of all four (the tiled layout keeps them together).
// The warps of a CTA take the chunks of k in turn, their sums are added in order through shared memory: the
// order of a sum depends on k alone, so a row's bits do not depend on the other rows.
#include <algorithm>

#include "block128.cuh"

namespace fme {

namespace {

constexpr int kGemvWarps = 8;
constexpr int kGemvThreads = 32 * kGemvWarps;
constexpr int kChunk = 128;  // k of a warp's step

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Eight codes of a word times their scale: pairs (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ void decode8(uint32_t w, uint32_t scale, uint32_t (&out)[4]) {
  const uint32_t v = w >> 8;
  out[0] = mul_bf16x2(((w & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, scale);
  out[1] = mul_bf16x2(((w & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, scale);
  out[2] = mul_bf16x2(((v & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, scale);
  out[3] = mul_bf16x2(((v & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, scale);
}

// Two E4M3 scales (the low 16 bits) times 2^118, each in both halves of a word.
__device__ __forceinline__ void decode_scales(uint32_t two, uint32_t (&out)[2]) {
  uint32_t h;
  asm("{\n\t.reg .b16 v;\n\tcvt.u16.u32 v, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, v;\n\t}" : "=r"(h) : "r"(two));
  float f0, f1;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f0), "=f"(f1)
      : "r"(h));
  f0 *= 0x1p118f;
  f1 *= 0x1p118f;
  asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(out[0]) : "f"(f0));
  asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(out[1]) : "f"(f1));
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load16(const void *p, bool ok) {
  return ok ? *static_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
}

struct Item {
  int32_t e;
  int32_t row0;    // first row of x (grouped)
  int32_t tokens;  // 1 .. 8 kBlocks
  int64_t w0;      // first weight row of unit 0's octet
};

// kBlocks token blocks of 8; kUnits groups of 32 weight rows (an octet of rows g in each quarter of 128): with kSwiglu
// the gate rows and the matching up rows, otherwise neighbouring octets.
template <int kBlocks, int kUnits, bool kSwiglu>
__global__ void __launch_bounds__(kGemvThreads, kBlocks == 4 ? 1 : 2) gemv_nvfp4_kernel(const __grid_constant__ LaunchGemv p) {
  constexpr int kTokens = 8 * kBlocks;
  constexpr int kRowsPad = 32 * kUnits + 1;
  extern __shared__ float dyn[];
  float *part = dyn;  // [warp][token][row]
  int32_t *off = reinterpret_cast<int32_t *>(dyn + kGemvWarps * kTokens * kRowsPad);
  int32_t *first = off + (p.num_experts + 1);
  __shared__ int ok_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  start_next_kernel();
  wait_for_previous_kernel();
  if (warp == 0) {
    const int32_t total = scan_groups(p.offsets, p.num_experts, p.m, kTokens,
                                      [&](int e, int32_t lo, int32_t, int32_t unit) {
                                        off[e] = lo;
                                        first[e] = unit;
                                      });
    if (lane == 0) {
      off[p.num_experts] = static_cast<int32_t>(p.m);
      first[p.num_experts] = total;
      ok_flag = total >= 0;
    }
  }
  __syncthreads();
  if (!ok_flag) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(p.status, kDevBadOffsets);
    return;
  }
  // Groups of 128 weight rows that an expert's rows lie in, and the items of each.
  const int64_t out_n = kSwiglu ? p.n / 2 : p.n;
  const int32_t blocks = static_cast<int32_t>(p.n % 128 == 0 ? out_n / 128 : (p.n + 254) / 128);
  constexpr int kPerBlock = kSwiglu ? 4 : 4 / kUnits;
  const uint32_t per = static_cast<uint32_t>(blocks) * kPerBlock;
  const uint32_t total = static_cast<uint32_t>(first[p.num_experts]) * per;
  const int32_t chunks = static_cast<int32_t>((p.k + kChunk - 1) / kChunk);
  const int64_t code_row = p.k / 2;

  auto item_at = [&](uint32_t i) {
    Item it;
    const uint32_t tile = i / per, u = i - tile * per;
    it.e = find_group(first, p.num_experts, tile);
    const int32_t skip = (static_cast<int32_t>(tile) - first[it.e]) * kTokens;
    it.row0 = off[it.e] + skip;
    it.tokens = min(kTokens, off[it.e + 1] - off[it.e] - skip);
    it.w0 = (((it.e * p.n) >> 7) + u / kPerBlock) * 128 + (u % kPerBlock) * (kSwiglu ? 8 : 8 * kUnits);
    return it;
  };
  // Weight row of unit u, lane row g, quarter q; rows of other experts count as absent.
  auto weight_row = [&](const Item &it, int u, int q) { return it.w0 + (kSwiglu ? u * out_n : 8 * u) + g + 32 * q; };
  auto present = [&](const Item &it, int64_t row) { return row >= it.e * p.n && row < (it.e + 1) * p.n; };

  struct Loads {
    uint4 code[kUnits][4];
    uint4 scale[kUnits];
  };
  auto load = [&](const Item &it, int32_t c, Loads &l) {
    const int64_t k0 = static_cast<int64_t>(c) * kChunk + t * 32;
    const bool in_k = c < chunks && k0 < p.k;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t row = weight_row(it, u, q);
        l.code[u][q] = load16(p.codes + row * code_row + k0 / 2, in_k && present(it, row));
      }
      const int64_t row = weight_row(it, u, 0);
      l.scale[u] = load16(p.sf + ((row >> 7) * (p.k >> 6) + (k0 >> 6)) * 512 + (row & 31) * 16,
                          in_k && (row >> 7) * 128 < p.num_experts * p.n);
    }
  };

  if (blockIdx.x >= total) return;
  Item it = item_at(blockIdx.x);
  Loads cur;
  load(it, warp, cur);
  for (uint32_t i = blockIdx.x; i < total; i += gridDim.x) {
    const uint32_t following = i + gridDim.x;
    Item next = it;
    if (following < total) next = item_at(following);
    // this lane's rows of x
    const uint16_t *xrow[kBlocks];
    bool live[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      live[b] = 8 * b + g < it.tokens;
      int64_t row = it.row0 + 8 * b + g;
      if (p.src_row != nullptr && live[b]) {
        const int32_t a = p.src_row[row];
        const bool fine = a >= 0 && a / p.top_k < p.x_rows;
        if (!fine && t == 0 && warp == 0) report(p.status, kDevBadIndex);
        row = fine ? a / p.top_k : 0;
      }
      xrow[b] = static_cast<const uint16_t *>(p.x) + row * p.k;
    }
    float acc[kUnits][2][kBlocks][4];
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[u][m][b][j] = 0.0f;

    for (int32_t c = warp; c < chunks; c += kGemvWarps) {
      Loads after;
      if (c + kGemvWarps < chunks)
        load(it, c + kGemvWarps, after);
      else if (following < total)
        load(next, warp, after);
      const int64_t k0 = static_cast<int64_t>(c) * kChunk + t * 32;
      uint32_t s[kUnits][4][2];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const uint32_t w[4] = {cur.scale[u].x, cur.scale[u].y, cur.scale[u].z, cur.scale[u].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) decode_scales(w[q] >> (16 * (t & 1)), s[u][q]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // 8 of the lane's 32 k
        uint32_t a[kUnits][4][4];
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 &v = cur.code[u][q];
            decode8(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w, s[u][q][j >> 1], a[u][q]);
          }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const uint4 x = load16(xrow[b] + k0 + 8 * j, live[b] && k0 < p.k);
          // the codes' pairs: (0, 4), (1, 5), (2, 6), (3, 7)
          const uint32_t b0 = __byte_perm(x.x, x.z, 0x5410), b1 = __byte_perm(x.x, x.z, 0x7632);
          const uint32_t b2 = __byte_perm(x.y, x.w, 0x5410), b3 = __byte_perm(x.y, x.w, 0x7632);
#pragma unroll
          for (int u = 0; u < kUnits; ++u)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              mma_16816(acc[u][m][b], a[u][2 * m][0], a[u][2 * m + 1][0], a[u][2 * m][1], a[u][2 * m + 1][1], b0, b1);
              mma_16816(acc[u][m][b], a[u][2 * m][2], a[u][2 * m + 1][2], a[u][2 * m][3], a[u][2 * m + 1][3], b2, b3);
            }
        }
      }
      cur = after;
    }
    if (warp >= chunks && following < total) load(next, warp, cur);  // (nothing: zeros)

    // ---- the warps' sums, in order
    float *mine = part + warp * kTokens * kRowsPad;
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mine[(8 * b + 2 * t + (j & 1)) * kRowsPad + 32 * u + 8 * (2 * m + (j >> 1)) + g] = acc[u][m][b][j];
    __syncthreads();
    constexpr int kOut = kSwiglu ? 32 : 32 * kUnits;  // outputs of a token
    for (int o = threadIdx.x; o < kOut * it.tokens; o += kGemvThreads) {
      const int tok = o / kOut, r = o % kOut;
      const int in_unit = r & 31;
      // rows of a unit: quarter r / 8, lane row r % 8
      const int64_t row = it.w0 + (kSwiglu ? 0 : 8 * (r >> 5)) + (in_unit & 7) + 32 * (in_unit >> 3);
      if (!present(it, row)) continue;
      float v = 0.0f, up = 0.0f;
      const int used = min(chunks, kGemvWarps);
      for (int w = 0; w < used; ++w) {
        v += part[(w * kTokens + tok) * kRowsPad + r];
        if (kSwiglu) up += part[(w * kTokens + tok) * kRowsPad + 32 + r];
      }
      v = (v * 256.0f) * p.scale[row];
      if (kSwiglu) v = silu_times(v, (up * 256.0f) * p.scale[row + out_n]);
      static_cast<__nv_bfloat16 *>(p.y)[(it.row0 + tok) * out_n + (row - it.e * p.n)] = __float2bfloat16_rn(v);
    }
    __syncthreads();
    it = next;
  }
}

template <int kBlocks, int kUnits, bool kSwiglu>
cudaError_t launch_gemv_as(const LaunchGemv &a) {
  auto kernel = gemv_nvfp4_kernel<kBlocks, kUnits, kSwiglu>;
  const int smem = kGemvWarps * 8 * kBlocks * (32 * kUnits + 1) * 4 + 8 * (a.num_experts + 1);
  static std::atomic<uint64_t> allowed{0};
  cudaError_t err = allow_shared(reinterpret_cast<const void *>(kernel), allowed);
  if (err != cudaSuccess) return err;
  const int64_t out_n = kSwiglu ? a.n / 2 : a.n;
  const int64_t per = (a.n % 128 == 0 ? out_n / 128 : (a.n + 254) / 128) * (kSwiglu ? 4 : 4 / kUnits);
  const int64_t items = (a.m / (8 * kBlocks) + std::min<int64_t>(a.num_experts, a.m)) * per;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>((kBlocks == 4 ? 1 : 2) * a.num_sms, items)), 1, 1);
  cfg.blockDim = dim3(kGemvThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_gemv_nvfp4(const LaunchGemv &a) {
  if (a.m <= 8 * static_cast<int64_t>(a.num_experts))
    return a.swiglu ? launch_gemv_as<1, 2, true>(a) : launch_gemv_as<1, 1, false>(a);
  if (a.m <= 16 * static_cast<int64_t>(a.num_experts))
    return a.swiglu ? launch_gemv_as<2, 2, true>(a) : launch_gemv_as<2, 2, false>(a);
  return a.swiglu ? launch_gemv_as<4, 2, true>(a) : launch_gemv_as<4, 2, false>(a);
}

}  // namespace fme
