// quant_block128.cu -- FP8 quantizers with one fp32 scale for each block of 128.
//
// For a block with largest magnitude a (over its non-NaN values):
//   A = max(a, 2^-100),  s = fl32(A / 448),  r = fl32(448 / A),  q = E4M3(fl32(x r)),
// round to nearest even, saturating at 448.  s is the stored scale.  The floor keeps
// r finite: a block of zeros gets codes 0 and a scale that dequantizes to 0.
// Row-wise blocks run along a row (the contraction of the forward and of dgrad),
// column-wise blocks along 128 padded token positions of one expert (the contraction
// of wgrad), weight blocks are 128 x 128 (both contractions read the same codes).
//
// Multiplying by r instead of dividing by s: two IEEE divisions a block instead of one
// an element; |x r| and |x / s| differ by at most 2^-22 of themselves, which moves a
// code only when it lies that close to the middle between two.
//
// All kernels are one pass, bound by HBM: 2 bytes read and 1 written (2 both ways) an
// element, plus 4 bytes a block.
#include "block128.cuh"

namespace fme {

namespace {

constexpr float kAmaxFloor = 7.8886090522101181e-31f;  // 2^-100

__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Largest magnitude of a word's two bf16, as bf16 bits; a half that has seen only NaN (which as an integer would
// be the largest) counts as 0.
__device__ __forceinline__ uint32_t absmax_halves(uint32_t m) {
  m = absmax2(m, 0u);
  return max(m & 0x7FFFu, (m >> 16) & 0x7FFFu);
}

struct BlockScale {
  float s, r;
};
// Both quotients correctly rounded, by one step of P. Markstein's fused-multiply-add refinement (IBM J.
// Res. Dev. 34(1), 1990): q + (n - d q) / d with the reciprocal in place of the last division.  A is
// taken times 2^-14 in the second, so that neither it nor its reciprocal leaves the normal range.
// Equal to IEEE division for every finite bf16 A from the floor up, and for reciprocals up to two ulps off
// (checked with exact rational arithmetic); two IEEE divisions a block were a fifth of the row-wise
// kernel's instructions.  An infinite A, for which the corrections are NaN, has its quotients set: inf and 0.
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
  const float a = fmaxf(bf16_bits_to_float(amax_bits), kAmaxFloor);
  constexpr float kInv = 1.0f / 448.0f;
  const float q = __fmul_rn(a, kInv);
  const float s = __fmaf_rn(__fmaf_rn(-448.0f, q, a), kInv, q);
  const float d = __fmul_rn(a, 0x1p-14f);
  const float t = rcp_approx(d);
  const float u = __fmul_rn(448.0f * 0x1p-14f, t);
  const float r = __fmaf_rn(__fmaf_rn(-d, u, 448.0f * 0x1p-14f), t, u);
  return a == INFINITY ? BlockScale{a, 0.0f} : BlockScale{s, r};
}

// The four bf16 of words a, b times (r0, r1, r2, r3) -> four E4M3 codes in order.
__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, float2 r01, float2 r23) {
  const float2 p = __fmul2_rn(make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u)), r01);
  const float2 q = __fmul2_rn(make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u)), r23);
  uint32_t w;
  asm("{\n\t.reg .b16 h0, h1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h0, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h1, %4, %3;\n\t"
      "mov.b32 %0, {h0, h1};\n\t}"
      : "=r"(w)
      : "f"(p.x), "f"(p.y), "f"(q.x), "f"(q.y));
  return w;
}

// ---------------------------------------------------------------- row-wise --
// One warp a row; a lane takes 16 consecutive values of every 512-wide chunk, eight
// lanes a block (three shuffles for its amax).  kUnroll chunks are loaded before they
// are coded.  gridDim.y splits a row's columns when there are few rows.  With
// `gather`, row r reads source row gather[r] / gather_div; an index outside
// [0, gather_limit) is reported and reads source row 0.
constexpr int kUnroll = 2;
constexpr int kChunkCols = 512;

template <bool kGather>
__global__ void __launch_bounds__(256) fp8_rows_kernel(const uint16_t *__restrict__ x, int64_t rows, int cols,
                                                       int cols_per_cta, uint8_t *__restrict__ codes,
                                                       float *__restrict__ scale, const int32_t *__restrict__ gather,
                                                       int gather_div, int64_t gather_limit, int32_t *status) {
  start_next_kernel();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  int64_t src = row;
  if constexpr (kGather) {
    const int32_t a = __ldg(gather + row);
    src = a / gather_div;
    if (a < 0 || src >= gather_limit) {
      if (lane == 0 && blockIdx.y == 0) report(status, kDevBadIndex);
      src = 0;
    }
  }
  const uint16_t *xr = x + src * cols;
  uint8_t *qr = codes + row * cols;
  const int c_lo = blockIdx.y * cols_per_cta;
  const int c_hi = min(cols, c_lo + cols_per_cta);
  for (int base = c_lo; base < c_hi; base += kUnroll * kChunkCols) {
    uint4 v[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int col = base + u * kChunkCols + lane * 16;
      v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
      if (col < c_hi) {
        v[u][0] = __ldg(reinterpret_cast<const uint4 *>(xr + col));
        v[u][1] = __ldg(reinterpret_cast<const uint4 *>(xr + col) + 1);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int col = base + u * kChunkCols + lane * 16;
      const uint4 a = v[u][0], b = v[u][1];
      uint32_t m = absmax2(absmax2(absmax2(a.x, a.y), absmax2(a.z, a.w)),
                           absmax2(absmax2(b.x, b.y), absmax2(b.z, b.w)));
      m = absmax2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = absmax2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      m = absmax2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
      const BlockScale f = block_scale(absmax_halves(m));
      const float2 r = make_float2(f.r, f.r);
      if (col < c_hi) {
        // streaming: the codes do not push the tokens out of L2
        __stcs(reinterpret_cast<uint4 *>(qr + col), make_uint4(codes4(a.x, a.y, r, r), codes4(a.z, a.w, r, r),
                                                               codes4(b.x, b.y, r, r), codes4(b.z, b.w, r, r)));
        if ((lane & 7) == 0) scale[static_cast<int64_t>(col >> 7) * rows + row] = f.s;
      }
    }
  }
}

// ------------------------------------------------- 128 x 128 tiles: the rest --
// A CTA holds a tile of 128 rows x 128 columns in registers: thread (rg, cg) has 8
// rows (8 rg ..) of 8 columns (8 cg ..), 16 lanes a row.  256 threads of 8 16-byte
// loads each, so that four to five CTAs an SM keep the loads in flight while others
// code.
//   kCols     column-wise codes and scales (and the padded offsets)
//   kRowCol   the same plus row-wise codes and scales, from one read
//   kWeights  one scale a tile
enum { kCols = 0, kRowCol = 1, kWeights = 2 };

template <int kMode>
__global__ void __launch_bounds__(256) fp8_tile_kernel(const uint16_t *__restrict__ x, int64_t rows, int cols,
                                                       const int32_t *__restrict__ offsets, int num_groups,
                                                       uint8_t *__restrict__ codes, float *__restrict__ scale,
                                                       int32_t *__restrict__ padded_offsets, int64_t chunks,
                                                       uint8_t *__restrict__ row_codes,
                                                       float *__restrict__ row_scale, int32_t *status) {
  __shared__ uint4 red[16][16];
  __shared__ float4 rcol[32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int cg = tid & 15, rg = tid >> 4;
  const int col_tiles = (cols + 127) >> 7;
  const int64_t chunk = blockIdx.x / col_tiles;  // of 128 padded positions (weights: of an expert's rows)
  const int ct = static_cast<int>(blockIdx.x - chunk * col_tiles);
  int64_t src0 = 0;   // first source row of the chunk
  int valid = 0;      // its rows
  if constexpr (kMode == kWeights) {  // rows = rows of one expert
    const int64_t per = (rows + 127) >> 7;
    const int64_t e = chunk / per, b = chunk - e * per;
    src0 = e * rows + b * 128;
    valid = static_cast<int>(min(int64_t(128), rows - b * 128));
  } else {
    // every warp finds the chunk's expert for itself
    int32_t found0 = 0, found_n = 0;
    const bool writer = padded_offsets != nullptr && blockIdx.x == 0 && tid < 32;
    const int32_t total =
        scan_groups(offsets, num_groups, rows, 128, [&](int g, int32_t lo, int32_t n, int32_t first) {
          const int64_t in = chunk - first;
          if (in >= 0 && in * 128 < n) {
            found0 = lo + static_cast<int32_t>(in * 128);
            found_n = min(128, n - static_cast<int32_t>(in * 128));
          }
          if (writer) {
            padded_offsets[g] = first * 128;
            if (g == num_groups - 1) padded_offsets[num_groups] = (first + (n > 0 ? (n + 127) / 128 : 0)) * 128;
          }
        });
    if (total < 0) {
      if (blockIdx.x == 0 && tid == 0) report(status, kDevBadOffsets);
      return;
    }
    if (chunk >= chunks) return;  // no positions at all: the offsets were all there was to write
    src0 = __reduce_add_sync(0xFFFFFFFFu, found0);  // one lane at most holds a chunk's rows
    valid = static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, found_n));
  }

  const int col = ct * 128 + cg * 8;
  const bool in_cols = col < cols;
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = rg * 8 + i;
    v[i] = make_uint4(0, 0, 0, 0);
    if (in_cols && r < valid) v[i] = __ldg(reinterpret_cast<const uint4 *>(x + (src0 + r) * cols + col));
  }

  if constexpr (kMode == kWeights) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = absmax2(m, absmax2(absmax2(v[i].x, v[i].y), absmax2(v[i].z, v[i].w)));
    const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, absmax_halves(m));
    uint32_t *part = reinterpret_cast<uint32_t *>(red);
    if (lane == 0) part[tid >> 5] = w;
    __syncthreads();
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, part[i]);
    const BlockScale f = block_scale(top);
    const float2 r2 = make_float2(f.r, f.r);
    if (tid == 0) scale[chunk * col_tiles + ct] = f.s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = rg * 8 + i;
      if (in_cols && r < valid)
        *reinterpret_cast<uint2 *>(codes + (src0 + r) * cols + col) =
            make_uint2(codes4(v[i].x, v[i].y, r2, r2), codes4(v[i].z, v[i].w, r2, r2));
    }
  } else {
    uint4 m = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m.x = absmax2(m.x, v[i].x);
      m.y = absmax2(m.y, v[i].y);
      m.z = absmax2(m.z, v[i].z);
      m.w = absmax2(m.w, v[i].w);
    }
    red[rg][cg] = m;
    __syncthreads();
    if (tid < 128) {  // thread = column
      const uint16_t *r16 = reinterpret_cast<const uint16_t *>(red) + tid;
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, static_cast<uint32_t>(r16[i * 128]) & 0x7FFFu);
      const BlockScale f = block_scale(top);
      reinterpret_cast<float *>(rcol)[tid] = f.r;
      if (ct * 128 + tid < cols) scale[chunk * cols + ct * 128 + tid] = f.s;
    }
    if constexpr (kMode == kRowCol) {
      // amax of this thread's 8 values of each of 8 rows, rows i and i + 4 in one
      // word; two shuffle steps leave a word a lane, two more reduce it over the rest
      // of the row's 16 lanes: lane l ends with row 2 (l & 1) + (l >> 1 & 1) + 4 (l >> 2 & 1)
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = absmax_halves(absmax2(absmax2(v[i].x, v[i].y), absmax2(v[i].z, v[i].w)));
        const uint32_t hi = absmax_halves(absmax2(absmax2(v[i + 4].x, v[i + 4].y), absmax2(v[i + 4].z, v[i + 4].w)));
        p[i] = lo | (hi << 16);
      }
      const bool b0 = lane & 1, b1 = lane & 2;
      const uint32_t k0 = b0 ? p[2] : p[0], k1 = b0 ? p[3] : p[1];
      const uint32_t s0 = b0 ? p[0] : p[2], s1 = b0 ? p[1] : p[3];
      const uint32_t q0 = absmax2(k0, __shfl_xor_sync(0xFFFFFFFFu, s0, 1));
      const uint32_t q1 = absmax2(k1, __shfl_xor_sync(0xFFFFFFFFu, s1, 1));
      uint32_t z = absmax2(b1 ? q1 : q0, __shfl_xor_sync(0xFFFFFFFFu, b1 ? q0 : q1, 2));
      z = absmax2(z, __shfl_xor_sync(0xFFFFFFFFu, z, 4));
      z = absmax2(z, __shfl_xor_sync(0xFFFFFFFFu, z, 8));
      const int mine = 2 * (lane & 1) + ((lane >> 1) & 1) + (lane & 4);
      const BlockScale f = block_scale((lane & 4) ? (z >> 16) & 0x7FFFu : z & 0x7FFFu);
      if (!(lane & 8) && rg * 8 + mine < valid) row_scale[ct * rows + src0 + rg * 8 + mine] = f.s;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float ri = __shfl_sync(0xFFFFFFFFu, f.r, (lane & 16) | ((i >> 1) & 1) | ((i & 1) << 1) | (i & 4));
        const float2 r2 = make_float2(ri, ri);
        const int r = rg * 8 + i;
        if (in_cols && r < valid)
          *reinterpret_cast<uint2 *>(row_codes + (src0 + r) * cols + col) =
              make_uint2(codes4(v[i].x, v[i].y, r2, r2), codes4(v[i].z, v[i].w, r2, r2));
      }
    }
    __syncthreads();
    const float4 ra = rcol[2 * cg], rb = rcol[2 * cg + 1];
    if (in_cols) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // padding positions hold zeros
        *reinterpret_cast<uint2 *>(codes + (chunk * 128 + rg * 8 + i) * cols + col) =
            make_uint2(codes4(v[i].x, v[i].y, make_float2(ra.x, ra.y), make_float2(ra.z, ra.w)),
                       codes4(v[i].z, v[i].w, make_float2(rb.x, rb.y), make_float2(rb.z, rb.w)));
      }
    }
  }
}

}  // namespace

cudaError_t launch_fp8_block128_rows(const LaunchFp8Quant &a) {
  const int64_t groups = (a.rows + 7) / 8;
  // few rows: split the columns (in steps of one pass) until there is a CTA for every SM
  const int steps = (a.cols + kUnroll * kChunkCols - 1) / (kUnroll * kChunkCols);
  int splits = 1;
  while (splits < steps && groups * splits < a.num_sms) ++splits;
  // a token's row is read once for each of its experts: 2048 columns of all rows at a time, so that
  // those columns of the tokens stay in L2 between (8192 tokens x 7168, top 8: 184 -> 147 us)
  if (a.gather_div > 1 && splits < (steps + 1) / 2) splits = (steps + 1) / 2;
  const int per = (steps + splits - 1) / splits * (kUnroll * kChunkCols);
  const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>((a.cols + per - 1) / per));
  auto kernel = a.gather ? fp8_rows_kernel<true> : fp8_rows_kernel<false>;
  kernel<<<grid, 256, 0, a.stream>>>(static_cast<const uint16_t *>(a.x), a.rows, static_cast<int>(a.cols), per, a.codes,
                                     a.scale, a.gather, a.gather_div, a.gather_limit, a.status);
  return cudaGetLastError();
}

template <int kMode>
static cudaError_t launch_tiles(const LaunchFp8Quant &a, int64_t chunks) {
  const int64_t tiles = chunks > 0 ? chunks * ((a.cols + 127) / 128) : 1;
  fp8_tile_kernel<kMode><<<static_cast<unsigned>(tiles), 256, 0, a.stream>>>(
      static_cast<const uint16_t *>(a.x), a.rows, static_cast<int>(a.cols), a.offsets, a.num_groups, a.codes, a.scale,
      a.padded_offsets, chunks, a.row_codes, a.row_scale, a.status);
  return cudaGetLastError();
}

cudaError_t launch_fp8_block128_cols(const LaunchFp8Quant &a) {
  return a.row_codes ? launch_tiles<kRowCol>(a, a.ld / 128) : launch_tiles<kCols>(a, a.ld / 128);
}

cudaError_t launch_fp8_block128_weights(const LaunchFp8Quant &a) {
  return launch_tiles<kWeights>(a, a.num_groups * ((a.rows + 127) / 128));
}

}  // namespace fme
