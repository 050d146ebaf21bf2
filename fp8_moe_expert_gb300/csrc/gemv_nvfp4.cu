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
// Any order of k will do as long as both operands follow it.  A unit is 32 weight rows: lane (g, t) = (lane / 4, lane % 4)
// of a warp takes 32 consecutive k of a chunk of 128 for four rows, g + 8 i of each quarter of a group of 128 (the tiled
// layout keeps the scales of those four together), or, with SwiGLU, of two quarters of the gate rows and of the matching
// up rows.  What a lane needs of a chunk, 16 bytes of codes a row and the scales, it copies itself into a ring in shared
// memory, some chunks ahead and across the ends of units, and reads back: no barrier, no conflict, and the loads in
// flight take no registers.  One, two, four or eight warps share a unit, by the length of k alone, each takes every
// such chunk, and their sums are added in order: the order of a sum depends on k alone, so a row's
// bits do not depend on the other rows.
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

// 16 or 8 bytes from global into shared memory, zeros where `bytes` is 0.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}

// A unit (or kUnits of them) and a tile of an expert's rows.  Weight rows, of all experts, are below 2^26.
struct Item {
  int32_t e;
  int32_t w0;    // its group of 128 weight rows
  int32_t part;  // which rows of it
  int32_t tile;  // tile of rows of x, of all experts
};

// kBlocks token blocks of 8, kUnits units of 32 weight rows, kShare warps to a unit's k, kDepth chunks in a warp's ring.
template <int kBlocks, int kUnits, bool kSwiglu, int kShare, int kDepth, int kCtas>
__global__ void __launch_bounds__(kGemvThreads, kCtas) gemv_nvfp4_kernel(const __grid_constant__ LaunchGemv p) {
  constexpr int kTokens = 8 * kBlocks;
  constexpr int kRowsPad = 32 * kUnits + 1;
  constexpr int kGroups = kGemvWarps / kShare;
  constexpr uint32_t kUnitBytes = 5 * 512;  // four rows' codes and their scales, 16 bytes a lane each
  constexpr uint32_t kSlotBytes = kUnits * kUnitBytes;
  extern __shared__ __align__(16) uint8_t dyn[];
  float *part = reinterpret_cast<float *>(dyn + kGemvWarps * kDepth * kSlotBytes);  // [warp][token][row]
  int32_t *off = reinterpret_cast<int32_t *>(part + kGemvWarps * kTokens * kRowsPad);
  int32_t *first = off + (p.num_experts + 1);
  __shared__ int ok_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int group = warp / kShare, share = warp % kShare;
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
  // Groups of 128 weight rows (with SwiGLU: gate rows) that an expert's rows lie in, and the items of each.
  const int32_t out_n = static_cast<int32_t>(kSwiglu ? p.n / 2 : p.n);
  const int32_t blocks = static_cast<int32_t>(p.n % 128 == 0 ? out_n / 128 : (p.n + 254) / 128);
  constexpr int kPerBlock = (kSwiglu ? 8 : 4) / kUnits;
  const uint32_t per = static_cast<uint32_t>(blocks) * kPerBlock;
  const uint32_t total = static_cast<uint32_t>(first[p.num_experts]) * per;
  const int32_t chunks = static_cast<int32_t>((p.k + kChunk - 1) / kChunk);
  const uint32_t stride = gridDim.x * kGroups;

  const int32_t n = static_cast<int32_t>(p.n);
  // Item i, the tile's expert looked for from expert e on.
  auto item_at = [&](uint32_t i, int32_t e) {
    Item it;
    const uint32_t tile = i / per, u = i - tile * per;
    while (first[e + 1] <= static_cast<int32_t>(tile)) ++e;
    it.e = e;
    it.tile = static_cast<int32_t>(tile);
    it.w0 = (((e * n) >> 7) + static_cast<int32_t>(u / kPerBlock)) * 128;
    it.part = static_cast<int32_t>(u % kPerBlock) * kUnits;
    return it;
  };
  // Weight row of lane row r, row slot q of unit u.  Plain: unit = octet of rows in each quarter, slot = quarter.
  // SwiGLU: unit = half of the quarters and octet, slots 0 and 1 gate rows of its two quarters, 2 and 3 the up rows.
  auto weight_row = [&](const Item &it, int u, int q, int r) {
    const int part_u = it.part + u;
    if (kSwiglu) return it.w0 + (q >> 1) * out_n + 32 * (2 * (part_u & 1) + (q & 1)) + 8 * (part_u >> 1) + r;
    return it.w0 + 32 * q + 8 * part_u + r;
  };
  auto present = [&](const Item &it, int32_t row) { return row >= it.e * n && row < (it.e + 1) * n; };

  // ---- copies: a cursor that runs kDepth chunks ahead of the sums
  const uint8_t *code[kUnits][4];
  const uint8_t *scale[kUnits][kSwiglu ? 2 : 1];
  uint32_t copy_item = blockIdx.x + gridDim.x * group;
  int32_t copy_c = share;
  int32_t copy_e = 0;
  auto aim = [&] {  // the addresses of copy_item's chunk copy_c
    const Item it = item_at(copy_item, copy_e);
    copy_e = it.e;
    const int32_t k0 = copy_c * kChunk + t * 32;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        int32_t row = weight_row(it, u, q, g);
        if (!present(it, row)) row = it.e * n;  // another expert's or none: any row, its sums are not used
        code[u][q] = p.codes + row * (p.k / 2) + k0 / 2;
      }
#pragma unroll
      for (int h = 0; h < (kSwiglu ? 2 : 1); ++h) {
        const int32_t row = weight_row(it, u, 2 * h, g);
        const int64_t blk = min(row >> 7, ((it.e + 1) * n - 1) >> 7);
        scale[u][h] = p.sf + (blk * (p.k >> 6) + (k0 >> 6)) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4;
      }
    }
  };
  const uint32_t ring = smem_u32(dyn) + warp * (kDepth * kSlotBytes) + lane * 16;
  auto copy_next = [&](uint32_t slot) {
    if (copy_item < total) {
      const uint32_t bytes = copy_c * kChunk + t * 32 < p.k ? 16u : 0u;
      const uint32_t to = ring + slot * kSlotBytes;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
#pragma unroll
        for (int q = 0; q < 4; ++q) copy16(to + u * kUnitBytes + q * 512, code[u][q], bytes);
        if (kSwiglu) {
          copy8(to + u * kUnitBytes + 4 * 512, scale[u][0], bytes >> 1);
          copy8(to + u * kUnitBytes + 4 * 512 + 8, scale[u][kSwiglu ? 1 : 0], bytes >> 1);
        } else {
          copy16(to + u * kUnitBytes + 4 * 512, scale[u][0], bytes);
        }
      }
      copy_c += kShare;
      if (copy_c < chunks) {
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
#pragma unroll
          for (int q = 0; q < 4; ++q) code[u][q] += kShare * (kChunk / 2);
#pragma unroll
          for (int h = 0; h < (kSwiglu ? 2 : 1); ++h) scale[u][h] += kShare * (kChunk / 64) * 512;
        }
      } else {
        copy_item += stride;
        copy_c = share;
        if (copy_item < total) aim();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (share >= chunks) copy_item = total;  // no chunk for this warp
  if (copy_item < total) aim();
#pragma unroll
  for (int d = 0; d < kDepth - 1; ++d) copy_next(d);
  uint32_t slot = 0;

  int32_t e_now = 0;
  for (uint32_t i = blockIdx.x + gridDim.x * group; i < total; i += stride) {
    const Item it = item_at(i, e_now);
    e_now = it.e;
    const int32_t skip = (it.tile - first[it.e]) * kTokens;
    const int32_t row0 = off[it.e] + skip, tokens = min(kTokens, off[it.e + 1] - off[it.e] - skip);
    // this lane's rows of x; of tokens that are not there the first, whose sums are not used
    const uint16_t *xrow[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const bool live = 8 * b + g < tokens;
      int64_t row = row0 + (live ? 8 * b + g : 0);
      if (p.src_row != nullptr) {
        const int32_t a = p.src_row[row];
        const bool fine = a >= 0 && a / p.top_k < p.x_rows;
        if (!fine && t == 0 && share == 0) report(p.status, kDevBadIndex);
        row = fine ? a / p.top_k : 0;
      }
      xrow[b] = static_cast<const uint16_t *>(p.x) + row * p.k + share * kChunk + t * 32;
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

    // With one token block the x of the next chunk is loaded while this one's sums are made.
    constexpr bool kAhead = kBlocks == 1;
    uint4 xa[4];
    auto load_x = [&](int32_t c) {
      const bool in_k = c * kChunk + t * 32 < p.k;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        xa[j] = in_k ? *reinterpret_cast<const uint4 *>(xrow[0] + 8 * j) : make_uint4(0, 0, 0, 0);
      xrow[0] += kShare * kChunk;
    };
    if (kAhead) load_x(share);
    for (int32_t c = share; c < chunks; c += kShare) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
      const uint32_t from = ring + slot * kSlotBytes;
      uint4 codes[kUnits][4];
      uint32_t sc[kUnits][4][2];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
#pragma unroll
        for (int q = 0; q < 4; ++q) codes[u][q] = shared16(from + u * kUnitBytes + q * 512);
        const uint4 w = shared16(from + u * kUnitBytes + 4 * 512);
        decode_scales(w.x >> (16 * (t & 1)), sc[u][0]);
        decode_scales(w.y >> (16 * (t & 1)), sc[u][1]);
        decode_scales(w.z >> (16 * (t & 1)), sc[u][2]);
        decode_scales(w.w >> (16 * (t & 1)), sc[u][3]);
      }
      // the slot that the sums left a chunk ago is filled again
      copy_next(slot == 0 ? kDepth - 1 : slot - 1);
      slot = slot == kDepth - 1 ? 0 : slot + 1;
      uint4 xc[4];
      if (kAhead) {
#pragma unroll
        for (int j = 0; j < 4; ++j) xc[j] = xa[j];
        load_x(c + kShare);
      }
      const bool in_k = c * kChunk + t * 32 < p.k;  // (a last chunk of 64)
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // 8 of the lane's 32 k
        uint32_t a[kUnits][4][4];
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 &v = codes[u][q];
            decode8(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w, sc[u][q][j >> 1], a[u][q]);
          }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          uint4 x;
          if (kAhead)
            x = xc[j];
          else
            x = in_k ? *reinterpret_cast<const uint4 *>(xrow[b] + 8 * j) : make_uint4(0, 0, 0, 0);
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
      if (!kAhead) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) xrow[b] += kShare * kChunk;
      }
    }

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
    auto meet = [&] {
      if (kShare == 1)
        __syncwarp();
      else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * kShare) : "memory");
    };
    meet();
    constexpr int kOut = kSwiglu ? 16 * kUnits : 32 * kUnits;  // outputs of a token
    const float *theirs = part + group * kShare * kTokens * kRowsPad;
    for (int o = share * 32 + lane; o < kOut * tokens; o += 32 * kShare) {
      const int tok = o / kOut, r = o % kOut;
      const int u = r / (kOut / kUnits), in = r % (kOut / kUnits);  // slot in / 8, lane row in % 8
      const int32_t row = weight_row(it, u, in >> 3, in & 7);
      if (!present(it, row)) continue;
      const float *from = theirs + tok * kRowsPad + 32 * u + in;
      float v = 0.0f, up = 0.0f;
#pragma unroll
      for (int w = 0; w < kShare; ++w) {
        v += from[w * kTokens * kRowsPad];
        if (kSwiglu) up += from[w * kTokens * kRowsPad + 16];
      }
      v = (v * 256.0f) * p.scale[row];
      if (kSwiglu) v = silu_times(v, (up * 256.0f) * p.scale[row + out_n]);
      static_cast<__nv_bfloat16 *>(p.y)[static_cast<int64_t>(row0 + tok) * out_n + (row - it.e * n)] = __float2bfloat16_rn(v);
    }
    meet();
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int kBlocks, int kUnits, bool kSwiglu, int kShare, int kDepth, int kCtas>
cudaError_t launch_gemv_as(const LaunchGemv &a) {
  auto kernel = gemv_nvfp4_kernel<kBlocks, kUnits, kSwiglu, kShare, kDepth, kCtas>;
  const int smem = kGemvWarps * (kDepth * kUnits * 2560 + 8 * kBlocks * (32 * kUnits + 1) * 4) + 8 * (a.num_experts + 1);
  static std::atomic<uint64_t> allowed{0};
  cudaError_t err = allow_shared(reinterpret_cast<const void *>(kernel), allowed);
  if (err != cudaSuccess) return err;
  const int64_t out_n = kSwiglu ? a.n / 2 : a.n;
  const int64_t per = (a.n % 128 == 0 ? out_n / 128 : (a.n + 254) / 128) * ((kSwiglu ? 8 : 4) / kUnits);
  const int64_t items = (a.m / (8 * kBlocks) + std::min<int64_t>(a.num_experts, a.m)) * per;
  cudaLaunchConfig_t cfg = {};
  constexpr int kGroups = kGemvWarps / kShare;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(kCtas * a.num_sms, (items + kGroups - 1) / kGroups)), 1, 1);
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

template <bool kSwiglu, int kShare>
cudaError_t launch_gemv_shared(const LaunchGemv &a) {
  if (a.m <= 8 * static_cast<int64_t>(a.num_experts)) return launch_gemv_as<1, 1, kSwiglu, kShare, 4, 2>(a);
  if (a.m <= 16 * static_cast<int64_t>(a.num_experts)) return launch_gemv_as<2, 2, kSwiglu, kShare, 3, 1>(a);
  return launch_gemv_as<4, 2, kSwiglu, kShare, 3, 1>(a);
}

template <bool kSwiglu>
cudaError_t launch_gemv(const LaunchGemv &a) {
  return a.k > 2048 || a.n <= 4096 ? launch_gemv_shared<kSwiglu, 8>(a) : launch_gemv_shared<kSwiglu, 2>(a);
}

}  // namespace

cudaError_t launch_gemv_nvfp4(const LaunchGemv &a) { return a.swiglu ? launch_gemv<true>(a) : launch_gemv<false>(a); }

}  // namespace fme
