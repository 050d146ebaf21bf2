// gemv_nvfp4.cu -- products of few bf16 rows with NVFP4 expert weights, for decode steps.
//
//   y[t, n] = S[e, n] sum_k x[t, k] c[e, n, k] sf[e, n, k / 16]      (t a row of expert e)
//
// from the codes c (E2M1), block scales sf (E4M3) and row scales S (fp32) of quantize_nvfp4_pertoken, the same weights
// as grouped_gemm_fwd_nvfp4's, with activations that stay bf16 ("Composer 2 Technical Report", section 6.1, the
// NVFP4 variant of the forward; for a few rows the time is that of reading the weights, and quantizing the rows would save
// nothing).  With SwiGLU the gate and the matching up rows are taken together and h = silu(g) u leaves.
//
// An E2M1 code times an E4M3 scale has at most six significant bits and lies in 2^-10 .. 2688: exact in fp16 and in bf16.
// The weights become 16-bit fragments in registers, multiplied by mma.sync (m16n8k16, fp32 sums).  A
// warp-wide MMA fits here where tcgen05 does not: its A operand comes from registers, and with at most 8 rows (its
// N) the tensor work is small; decoding is what the SM spends its time on.  Two ways:
//   fp16  4 conversions and 4 products for the 8 codes of a word.  x, times a power of two that brings its row's largest
//         value to 2^14 .. 2^15, must be exact in fp16: a bf16 value is, down to 2^-29 of the largest;
//   bf16  where it is not (a row with a wider range or a NaN; one with an infinity is looked at unscaled): two codes of a
//         word lie 16 bits apart, one in each half.  A masked pair times (2^12 + 2^6) puts a code's sign into bit 15 and its
//         exponent and mantissa into bits 8 .. 6 of each half, as bf16 the code's value times 2^-126 (its subnormal 0.5 a bf16
//         subnormal).  Times sf 2^118 it is c sf 2^-8.  13 integer operations and 4 products for 8 codes.
// Both multiply the same values but for a power of two, so the sums' bits are the same (as long as they are normal
// numbers).  Gate/up of 4096 x 7168, 8 and all of 32 experts with a row each: 30 and 91 us (4.4 and 5.8 TB/s of weights), in
// bf16 38 and 121.
//
// Any order of k will do as long as both operands follow it.  A unit is 32 weight rows: 8 of each quarter of a group of 128
// (the tiled layout keeps the scales of rows 32 apart together), or, with SwiGLU, of two quarters of the gate rows
// and of the matching up rows.  A warp's step is a chunk of 256 k of a unit: four boxes of 8 rows x 128 bytes of codes and the
// tiles of scales come by bulk tensor copies into a ring of the warp's own, a step or two ahead and across the ends of units.
// Lane (g, t) = (lane / 4, lane % 4) takes 32 consecutive k of each half chunk for one row of each box.
//
// Two, four or eight warps share a unit, by how many there are.  The chunks of each residue mod 8
// have a sum of their own, and the eight are added as a tree, ((0 + 4) + (2 + 6)) + ((1 + 5) + (3 + 7)), of which each warp
// makes its branch: the order is the same however many warps share, so a row's bits do not depend on the other rows.
//
// A CTA an SM, 16 warps, takes consecutive units, mostly of the same up to 8 rows of x: those it brings into shared memory
// once, converted, in the order in which the lanes read them, several experts' together where they fit.  The most rows that any
// expert has decide how much of it they take, and so how deep the rings are.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "gemm_tiles.cuh"

namespace fme {

namespace {

constexpr int kGemvWarps = 16;
constexpr int kGemvThreads = 32 * kGemvWarps;
constexpr int kChunk = 256;    // k of a warp's step
constexpr int kRowsPad = 33;   // sums of a row of x in shared memory
constexpr uint32_t kBoxBytes = 8 * 128;    // 8 rows' codes of a chunk
constexpr uint32_t kCodeBytes = 4 * kBoxBytes;
constexpr uint32_t kTilesBytes = 4 * 128;  // scales of 8 rows of each quarter of a chunk
constexpr int kSums = 8;                  // of every output: one of each residue of the chunks mod 8
constexpr int kXPad = 64;                 // bytes between the rows of x, so that two of them cover all banks

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Eight codes of a word times their scale.  fp16: pairs (0, 1), (2, 3), (4, 5), (6, 7); bf16: (0, 4), (1, 5), (2, 6), (3, 7).
template <bool kHalf>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t scale, uint32_t (&out)[4]) {
  if constexpr (kHalf) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
        "mov.b32 {c0, c1, c2, c3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, c0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, c1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, c3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = mul_f16x2(h[i], scale);
  } else {
    const uint32_t v = w >> 8;
    out[0] = mul_bf16x2(((w & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, scale);
    out[1] = mul_bf16x2(((w & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, scale);
    out[2] = mul_bf16x2(((v & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, scale);
    out[3] = mul_bf16x2(((v & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, scale);
  }
}

// Two E4M3 scales (the low 16 bits), each in both halves of a word: as fp16, or times 2^118 as bf16.
template <bool kHalf>
__device__ __forceinline__ void decode_scales(uint32_t two, uint32_t (&out)[2]) {
  uint32_t h;
  asm("{\n\t.reg .b16 v;\n\tcvt.u16.u32 v, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, v;\n\t}" : "=r"(h) : "r"(two));
  if constexpr (kHalf) {
    out[0] = __byte_perm(h, h, 0x1010);
    out[1] = __byte_perm(h, h, 0x3232);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(out[0]) : "f"(f.x * 0x1p118f));
    asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(out[1]) : "f"(f.y * 0x1p118f));
  }
}

template <bool kHalf>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if constexpr (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}
__device__ __forceinline__ uint2 shared8(uint32_t src) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(src) : "memory");
  return v;
}

// Eight bf16 values as fp32.
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

struct SharedGemv {
  uint64_t full[kGemvWarps][2];
  float amax[kGemvWarps];       // of a warp's part of a row of x
  float back[kGemvRows];        // 2^-s of each row's power of two
  int ok_flag;
  int abort_flag;
  int x_tile;  // rows of x of the largest tile
};

// A unit's place.  Weight rows, of all experts, are below 2^26.
struct Unit {
  int32_t e;
  int32_t w0;    // its group of 128 weight rows
  int32_t part;  // which rows of it
};

template <bool kSwiglu, int kShare>
__global__ void __launch_bounds__(kGemvThreads, 1) gemv_nvfp4_kernel(const __grid_constant__ LaunchGemv p) {
  constexpr int kGroups = kGemvWarps / kShare;
  constexpr int kSets = kSums / kShare;  // of the eight sums, a warp's
  constexpr uint32_t kScaleBytes = (kSwiglu ? 2 : 1) * kTilesBytes;
  __shared__ SharedGemv s;
  extern __shared__ uint8_t dyn_smem[];
  uint8_t *dyn = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  const int32_t k = static_cast<int32_t>(p.k), n = static_cast<int32_t>(p.n);
  const int32_t chunks = (k + kChunk - 1) / kChunk;
  const uint32_t x_stride = chunks * kChunk * 2 + kXPad;  // bytes of a row of x
  int32_t *off = reinterpret_cast<int32_t *>(dyn);
  int32_t *first = off + (p.num_experts + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the row of a box that the lane takes: lanes of one phase of an access to shared memory read rows 4 apart, which the
  // swizzle keeps in different banks
  const int g = (lane >> 3) | (((lane >> 2) & 1) << 2), t = lane & 3;
  const int group = warp / kShare, share = warp % kShare;
  if (lane == 0) {
    mbar_init(&s.full[warp][0], 1);
    mbar_init(&s.full[warp][1], 1);
    if (warp == 0) {
      s.abort_flag = 0;
      prefetch_tensormap(&p.map_codes);
      prefetch_tensormap(&p.map_sf);
    }
    fence_barrier_init();
    fence_proxy_async_shared();
  }
  start_next_kernel();
  wait_for_previous_kernel();
  if (warp == 0) {
    int32_t most = 0;
    const int32_t total = scan_groups(p.offsets, p.num_experts, p.m, p.tile_rows,
                                      [&](int e, int32_t lo, int32_t rows, int32_t unit) {
                                        off[e] = lo;
                                        first[e] = unit;
                                        most = max(most, rows);
                                      });
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) {
      off[p.num_experts] = static_cast<int32_t>(p.m);
      first[p.num_experts] = total;
      s.ok_flag = total >= 0;
      s.x_tile = min(most, p.tile_rows);
    }
  }
  __syncthreads();
  if (!s.ok_flag) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(p.status, kDevBadOffsets);
    return;
  }
  // the rings, the warps' sums, the rows of x: two chunks a warp and two buffers of sums where they fit beside the rows of the
  // largest tile
  constexpr uint32_t kPartBytes = kGemvWarps * kGemvRows * kRowsPad * 4;
  constexpr uint32_t kRingBytes = kGemvWarps * (kCodeBytes + kScaleBytes);
  const uint32_t ring_off = (8 * (p.num_experts + 1) + 1023) & ~1023u;
  const uint32_t least = ring_off + kRingBytes + kPartBytes + s.x_tile * x_stride;
  const int depth = least + kRingBytes <= p.shared_bytes ? 2 : 1;
  const bool two_parts = least + (depth - 1) * kRingBytes + kPartBytes <= p.shared_bytes;
  uint8_t *codes_ring = dyn + ring_off + warp * depth * kCodeBytes;
  uint8_t *scales_ring = dyn + ring_off + kGemvWarps * depth * kCodeBytes + warp * depth * kScaleBytes;
  float *part = reinterpret_cast<float *>(dyn + ring_off + depth * kRingBytes);  // [buffer][warp][row of x][weight row]
  const uint32_t xs_off = ring_off + depth * kRingBytes + (two_parts ? 2 : 1) * kPartBytes;
  uint8_t *xs = dyn + xs_off;
  // Groups of 128 weight rows (with SwiGLU: gate rows) that an expert's rows lie in, and the units of each.
  const int32_t out_n = kSwiglu ? n / 2 : n;
  const int32_t blocks = n % 128 == 0 ? out_n / 128 : (n + 254) / 128;
  constexpr int kPerBlock = kSwiglu ? 8 : 4;
  const uint32_t per = static_cast<uint32_t>(blocks) * kPerBlock;  // units of a tile of rows of x
  const uint32_t total = static_cast<uint32_t>(first[p.num_experts]) * per;
  // this CTA's units
  const uint32_t begin = static_cast<uint32_t>(static_cast<uint64_t>(total) * blockIdx.x / gridDim.x);
  const uint32_t end = static_cast<uint32_t>(static_cast<uint64_t>(total) * (blockIdx.x + 1) / gridDim.x);

  if (begin == end) return;

  // The expert of a tile, from the expert of an earlier one.
  auto expert_of = [&](uint32_t tile, int32_t e) {
    if (first[e + 1] > static_cast<int32_t>(tile)) return e;
    return e + 1 + find_group(first + e + 1, p.num_experts - e - 1, tile);
  };
  // Unit i of tile `tile` of expert e.
  auto unit_at = [&](uint32_t i, uint32_t tile, int32_t e) {
    const int32_t u = static_cast<int32_t>(i - tile * per);
    return Unit{e, (((e * n) >> 7) + u / kPerBlock) * 128, u % kPerBlock};
  };
  // Weight row of lane row r, row slot q.  Plain: a unit is an octet of rows in each quarter, a slot a quarter.
  // SwiGLU: it is half of the quarters and an octet, slots 0 and 1 gate rows of its two quarters, 2 and 3 the up rows.
  auto weight_row = [&](const Unit &it, int q, int r) {
    if (kSwiglu) return it.w0 + (q >> 1) * out_n + 32 * (2 * (it.part & 1) + (q & 1)) + 8 * (it.part >> 1) + r;
    return it.w0 + 32 * q + 8 * it.part + r;
  };
  auto present = [&](const Unit &it, int32_t row) { return row >= it.e * n && row < (it.e + 1) * n; };

  // ---- copies of the weights, by lane 0: a cursor that runs `depth` chunks ahead of the sums
  volatile int *abort_flag = &s.abort_flag;
  uint32_t copy_unit = share < chunks ? begin + group : end, filled = 0;
  int32_t e = find_group(first, p.num_experts, begin / per), copy_c = share, copy_e = e;
  Unit copy{};
  auto aim = [&] {
    const uint32_t tile = copy_unit / per;
    copy_e = expert_of(tile, copy_e);
    copy = unit_at(copy_unit, tile, copy_e);
  };
  auto copy_next = [&](int slot) {
    if (lane == 0 && copy_unit < end) {
      uint64_t *bar = &s.full[warp][slot];
      mbar_arrive_expect_tx(bar, kCodeBytes + kScaleBytes);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        tma_load_2d_own(codes_ring + slot * kCodeBytes + q * kBoxBytes, &p.map_codes, bar, copy_c * (kChunk / 2),
                        weight_row(copy, q, 0));
#pragma unroll
      for (int h = 0; h < (kSwiglu ? 2 : 1); ++h) {
        const int32_t row = weight_row(copy, 2 * h, 0);
        tma_load_3d_own(scales_ring + slot * kScaleBytes + h * kTilesBytes, &p.map_sf, bar, (row & 31) * 16,
                        copy_c * (kChunk / 64), row >> 7);
      }
      ++filled;
      copy_c += kShare;
      if (copy_c >= chunks) {
        copy_unit += kGroups;
        copy_c = share;
        if (copy_unit < end) aim();
      }
    }
    __syncwarp();
  };
  if (copy_unit < end) aim();
  for (int d = 0; d < depth; ++d) copy_next(d);
  uint32_t used = 0;  // chunks so far

  const uint32_t xs_at = smem_u32(xs);
  // The rows of a tile of expert e.
  auto row_of = [&](uint32_t tile, int32_t e) { return off[e] + (static_cast<int32_t>(tile) - first[e]) * p.tile_rows; };
  auto row_end = [&](uint32_t tile, int32_t e) { return min(row_of(tile, e) + p.tile_rows, off[e + 1]); };
  uint32_t i = begin + group, turn = 0;
  for (uint32_t tile = begin / per, next; tile * per < end; tile = next) {
    // ---- a pass: the tile and those behind it, as far as this CTA has units of them and there is room for their rows (their
    // units then run side by side: 16 of 32 experts of 7168 x 2048 with a row each 30.0 us, one tile after the other 33.0)
    e = expert_of(tile, e);
    const int32_t row0 = row_of(tile, e);
    int32_t rows = row_end(tile, e) - row0;
    next = tile + 1;
    if (next * per < end) {
      const int32_t room = min(kGemvRows, static_cast<int32_t>((p.shared_bytes - xs_off) / x_stride));
      for (int32_t last_e = e; next * per < end; ++next) {
        last_e = expert_of(next, last_e);
        const int32_t more = row_end(next, last_e) - row0;
        if (more > room) break;
        rows = more;
      }
    }

    // ---- its rows of x: the power of two of each, then their values in the order in which the lanes read them.
    // 16 / 2^j warps to a row.
    const int per_row = rows == 1 ? 16 : rows == 2 ? 8 : rows <= 4 ? 4 : 2;
    const int mine = warp / per_row, slice = warp % per_row;
    const uint16_t *src = nullptr;
    if (mine < rows) {
      int64_t row = row0 + mine;
      if (p.src_row != nullptr) {
        const int32_t a = p.src_row[row];
        const bool fine = a >= 0 && a / p.top_k < p.x_rows;
        if (!fine && lane == 0) report(p.status, kDevBadIndex);
        row = fine ? a / p.top_k : 0;
      }
      src = static_cast<const uint16_t *>(p.x) + row * k;
      float top = 0.0f;
      for (int c = slice * 32 + lane; c < k / 8; c += 4 * per_row * 32) {
        uint4 v[4];
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (c + b * per_row * 32 < k / 8) v[b] = *reinterpret_cast<const uint4 *>(src + 8 * (c + b * per_row * 32));
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (c + b * per_row * 32 >= k / 8) continue;
          float f[8];
          unpack8(v[b], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(f[j]));
        }
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      if (lane == 0) s.amax[warp] = top;
    }
    __syncthreads();  // also: the pass before is no longer read
    float power = 1.0f;
    if (mine < rows) {
      float top = s.amax[mine * per_row];
      for (int j = 1; j < per_row; ++j) top = fmaxf(top, s.amax[mine * per_row + j]);
      // 2^s, s = 14 - the exponent of the largest, at most 120 (0 and infinity: any)
      const int exponent = static_cast<int>(__float_as_uint(top) >> 23);
      const int shift = exponent == 255 ? 0 : min(14 - (exponent - 127), 120);
      power = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
      if (slice == 0 && lane == 0) s.back[mine] = __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
    }
    auto place = [&](bool half) {
      bool exact = true;
      for (int c = slice * 32 + lane; c < chunks * (kChunk / 8); c += per_row * 32) {
        uint4 v = make_uint4(0, 0, 0, 0);  // behind k
        if (c < k / 8) v = *reinterpret_cast<const uint4 *>(src + 8 * c);
        uint4 o;
        if (half) {
          float f[8];
          unpack8(v, f);
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float lo = f[2 * j] * power, hi = f[2 * j + 1] * power;
            const __half2 h = __floats2half2_rn(lo, hi);
            const float2 b = __half22float2(h);
            exact = exact && b.x == lo && b.y == hi && (lo != 0.0f || f[2 * j] == 0.0f) && (hi != 0.0f || f[2 * j + 1] == 0.0f);
            w[j] = *reinterpret_cast<const uint32_t *>(&h);
          }
          o = make_uint4(w[0], w[1], w[2], w[3]);
        } else {  // the pairs of the bf16 codes
          o = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                         __byte_perm(v.y, v.w, 0x7632));
        }
        // piece c = 16 half + 4 t + j of the row goes where the lanes t = 0 .. 3 read their j-th side by side
        const int at = (c & ~15) + 4 * (c & 3) + ((c >> 2) & 3);
        *reinterpret_cast<uint4 *>(xs + mine * x_stride + 16 * at) = o;
      }
      return exact;
    };
    const bool wide = __syncthreads_or(mine < rows && !place(true)) != 0;  // some row is not exact in fp16
    if (wide) {
      if (mine < rows) place(false);
      __syncthreads();
    }
    // (rows of x that are not there: the first, whose sums are not used)
    const uint32_t x_lane = xs_at + (lane / 4 < rows ? lane / 4 : 0) * x_stride + t * 16;

    // ---- its units
    for (uint32_t of = tile; of < next; ++of) {
      e = expert_of(of, e);
      const int32_t from_row = row_of(of, e) - row0, to_row = row_end(of, e) - row0;
      const uint32_t stop = min(end, (of + 1) * per);
      for (; i < stop; i += kGroups, ++turn) {
        const Unit it = unit_at(i, of, e);
        const uint32_t quarters = kSwiglu ? (it.part & 1) * 8 : 0;  // SwiGLU: its two words of a row's four
        // the weight row whose outputs this lane will write, and its scales, on their way while the sums are made
        constexpr int kOut = kSwiglu ? 16 : 32;  // outputs of a row of x
        const int out = lane % kOut;             // slot out / 8, lane row out % 8
        const int32_t out_row = weight_row(it, out >> 3, out & 7);
        const bool writes = present(it, out_row);
        const float scale = writes ? p.scale[out_row] : 0.0f;
        const float up_scale = kSwiglu && writes ? p.scale[out_row + out_n] : 0.0f;
        float acc[kSets][2][4] = {};
        auto sums = [&](auto half_tag) {
          constexpr bool kHalf = decltype(half_tag)::value;
          auto add_chunk = [&](int32_t c, float(&sum)[2][4]) {
            const int slot = depth == 2 ? used & 1 : 0;
            // (a wait that ran out: garbage from here on, which is not stored, and no more copies)
            if (!mbar_wait(&s.full[warp][slot], (depth == 2 ? used >> 1 : used) & 1, abort_flag, p.status)) copy_unit = end;
            __syncwarp();
            ++used;
            const uint32_t boxes = smem_u32(codes_ring) + slot * kCodeBytes + g * 128;
            const uint32_t tiles = smem_u32(scales_ring) + slot * kScaleBytes + (t >> 1) * 128 + g * 16 + quarters;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint4 codes[4], w;  // w: the words of the four rows' scales
#pragma unroll
              for (int q = 0; q < 4; ++q) codes[q] = shared16(boxes + q * kBoxBytes + (((4 * half + t) ^ g) * 16));
              if (kSwiglu) {
                const uint2 gate = shared8(tiles + half * 256), up = shared8(tiles + half * 256 + kTilesBytes);
                w = make_uint4(gate.x, gate.y, up.x, up.y);
              } else {
                w = shared16(tiles + half * 256);
              }
              if (half == 1) {  // all of the slot is read: its next chunk may be on its way
                asm volatile("" ::"r"(codes[3].w), "r"(w.w) : "memory");
                __syncwarp();
                copy_next(slot);
              }
              const int32_t k0 = c * kChunk + half * 128;
              if (k0 >= k) continue;
              uint32_t sc[4][2];
              decode_scales<kHalf>(w.x >> (16 * (t & 1)), sc[0]);
              decode_scales<kHalf>(w.y >> (16 * (t & 1)), sc[1]);
              decode_scales<kHalf>(w.z >> (16 * (t & 1)), sc[2]);
              decode_scales<kHalf>(w.w >> (16 * (t & 1)), sc[3]);
#pragma unroll
              for (int j = 0; j < 4; ++j) {  // 8 of the lane's 32 k
                uint32_t a[4][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const uint4 &v = codes[q];
                  decode8<kHalf>(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w, sc[q][j >> 1], a[q]);
                }
                const uint4 x = shared16(x_lane + k0 * 2 + 64 * j);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                  mma_16816<kHalf>(sum[m], a[2 * m][0], a[2 * m + 1][0], a[2 * m][1], a[2 * m + 1][1], x.x, x.y);
                  mma_16816<kHalf>(sum[m], a[2 * m][2], a[2 * m + 1][2], a[2 * m][3], a[2 * m + 1][3], x.z, x.w);
                }
              }
            }
          };
          for (int32_t c = share; c < chunks; c += kSums) {
#pragma unroll
            for (int set = 0; set < kSets; ++set)
              if (c + set * kShare < chunks) add_chunk(c + set * kShare, acc[set]);
          }
        };
        if (wide)
          sums(std::false_type{});
        else
          sums(std::true_type{});

        // ---- the eight sums: a warp's own, then the warps'
        if constexpr (kSets > 1) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[0][m][j] = kSets == 2 ? acc[0][m][j] + acc[1][m][j]
                                        : (acc[0][m][j] + acc[kSets / 2][m][j]) + (acc[1][m][j] + acc[kSets - 1][m][j]);
        }
        // With two buffers in turn a warp writes one again only after the others, done with it, have met once more: 56 -> 53 us
        // for the down projection of all 32 experts.
        float *sums_of = part + (two_parts ? turn & 1 : 0) * (kPartBytes / 4);
        float *to_part = sums_of + warp * kGemvRows * kRowsPad;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) to_part[(2 * t + (j & 1)) * kRowsPad + 8 * (2 * m + (j >> 1)) + g] = acc[0][m][j];
        auto meet = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * kShare) : "memory"); };
        meet();
        const bool garbage = *abort_flag != 0;  // some warp's sums
        const float *theirs = sums_of + group * kShare * kGemvRows * kRowsPad + out;
        for (int tok = from_row + (share * 32 + lane) / kOut; tok < to_row && writes && !garbage; tok += 32 * kShare / kOut) {
          const float *from = theirs + tok * kRowsPad;
          auto joined = [&](const float *at) {
            float w[kShare];
#pragma unroll
            for (int j = 0; j < kShare; ++j) w[j] = at[j * kGemvRows * kRowsPad];
#pragma unroll
            for (int half = kShare / 2; half; half /= 2)
#pragma unroll
              for (int j = 0; j < half; ++j) w[j] += w[j + half];
            return w[0];
          };
          float v = joined(from);
          const float up = kSwiglu ? joined(from + 16) : 0.0f;
          const float back = wide ? 256.0f : s.back[tok];
          v = (v * back) * scale;
          if (kSwiglu) v = silu_times(v, (up * back) * up_scale);
          static_cast<__nv_bfloat16 *>(p.y)[static_cast<int64_t>(row0 + tok) * out_n + (out_row - it.e * n)] =
              __float2bfloat16_rn(v);
        }
        if (!two_parts) meet();
      }
    }
  }
  // A wait that ran out leaves copies behind: they land before the CTA can exit.
  if (lane == 0)
    for (uint32_t f = filled > static_cast<uint32_t>(depth) ? filled - depth : 0; f < filled; ++f)
      mbar_drain(&s.full[warp][depth == 2 ? f & 1 : 0], (depth == 2 ? f >> 1 : f) & 1);
}

template <bool kSwiglu, int kShare>
cudaError_t launch_gemv(LaunchGemv a) {
  auto kernel = gemv_nvfp4_kernel<kSwiglu, kShare>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t err = allow_shared(reinterpret_cast<const void *>(kernel), allowed);
  if (err != cudaSuccess) return err;
  a.tile_rows = gemv_tile_rows(a.k);
  // all the shared memory of an SM: how it is used follows from the rows of the experts
  a.shared_bytes = 226 * 1024 - (sizeof(SharedGemv) + 127) / 128 * 128;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(a.num_sms, gemv_units(a.swiglu, a.m, a.n, a.k, a.num_experts))), 1, 1);
  cfg.blockDim = dim3(kGemvThreads, 1, 1);
  cfg.dynamicSmemBytes = a.shared_bytes + 1024;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool kSwiglu>
cudaError_t launch_gemv(const LaunchGemv &a) {
  switch (gemv_share(gemv_units(a.swiglu, a.m, a.n, a.k, a.num_experts), a.k, a.num_sms)) {
    case 8: return launch_gemv<kSwiglu, 8>(a);
    case 4: return launch_gemv<kSwiglu, 4>(a);
    default: return launch_gemv<kSwiglu, 2>(a);
  }
}

}  // namespace

cudaError_t launch_gemv_nvfp4(const LaunchGemv &a) { return a.swiglu ? launch_gemv<true>(a) : launch_gemv<false>(a); }

}  // namespace fme
