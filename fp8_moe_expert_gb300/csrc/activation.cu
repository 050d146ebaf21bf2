// activation.cu -- SwiGLU between the projections in bf16, forward and backward.
//
//   h = silu(g) * u,   dg = dh * u * sigma(g) * (1 + g * sigma(-g)),   du = dh * g * sigma(g)
//
// for rows [g | u] of the gate/up projection, each in fp32 and rounded once; the bits of the activation that
// swiglu_quantize_nvfp4 and swiglu_backward_quantize_mxfp8 quantize.  One pass: 6 bytes an element forward, 10 backward, bound
// by memory: 65536 x 2048, 115 us (7.0 TB/s) and 188 us (7.1 TB/s).  A CTA takes 1024 pieces of 8 elements, four to a
// thread, all loads before the first use.
#include "block128.cuh"
#include "swiglu.cuh"

namespace fme {

namespace {

constexpr int kActThreads = 256;
constexpr int kActPieces = 4;

template <bool kBackward>
__global__ void __launch_bounds__(kActThreads) swiglu_kernel(const uint16_t *gate_up, const uint16_t *dh, int64_t pieces,
                                                             uint32_t per_row, uint16_t *out) {
  start_next_kernel();
  wait_for_previous_kernel();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kActThreads * kActPieces);
  const int64_t row0 = base / per_row;
  const uint32_t at0 = static_cast<uint32_t>(base - row0 * per_row);
  uint4 g[kActPieces], u[kActPieces], d[kActPieces];
  int64_t wide[kActPieces], narrow[kActPieces];  // element offsets in rows of 2 inter and of inter
  bool ok[kActPieces];
#pragma unroll
  for (int i = 0; i < kActPieces; ++i) {
    const uint32_t j = threadIdx.x + i * kActThreads, at = at0 + j;
    ok[i] = base + j < pieces;
    const int64_t row = row0 + at / per_row;
    const int64_t col = static_cast<int64_t>(at % per_row) * 8;
    wide[i] = row * per_row * 16 + col;
    narrow[i] = row * per_row * 8 + col;
    if (!ok[i]) continue;
    g[i] = *reinterpret_cast<const uint4 *>(gate_up + wide[i]);
    u[i] = *reinterpret_cast<const uint4 *>(gate_up + wide[i] + static_cast<int64_t>(per_row) * 8);
    if (kBackward) d[i] = *reinterpret_cast<const uint4 *>(dh + narrow[i]);
  }
#pragma unroll
  for (int i = 0; i < kActPieces; ++i) {
    if (!ok[i]) continue;
    if (kBackward) {
      uint4 dg, du;
      swiglu_bwd_uint4(g[i], u[i], d[i], dg, du);
      *reinterpret_cast<uint4 *>(out + wide[i]) = dg;
      *reinterpret_cast<uint4 *>(out + wide[i] + static_cast<int64_t>(per_row) * 8) = du;
    } else {
      *reinterpret_cast<uint4 *>(out + narrow[i]) = swiglu_uint4(g[i], u[i]);
    }
  }
}

}  // namespace

cudaError_t launch_swiglu(const LaunchSwiglu &a) {
  const int64_t pieces = a.rows * (a.inter / 8);
  const uint32_t per_row = static_cast<uint32_t>(a.inter / 8);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((pieces + kActThreads * kActPieces - 1) / (kActThreads * kActPieces)), 1, 1);
  cfg.blockDim = dim3(kActThreads, 1, 1);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const uint16_t *gu = static_cast<const uint16_t *>(a.gate_up), *dh = static_cast<const uint16_t *>(a.dh);
  return a.dh ? cudaLaunchKernelEx(&cfg, swiglu_kernel<true>, gu, dh, pieces, per_row, static_cast<uint16_t *>(a.out))
              : cudaLaunchKernelEx(&cfg, swiglu_kernel<false>, gu, dh, pieces, per_row, static_cast<uint16_t *>(a.out));
}

}  // namespace fme
