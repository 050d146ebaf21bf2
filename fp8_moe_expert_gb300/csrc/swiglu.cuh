// swiglu.cuh -- h = silu(g) * u and its gradient on bf16 words, shared by the quantizers that fuse it and by
// activation.cu, so that all of them form the same bits.
#pragma once

#include "fme_device.cuh"

namespace fme {

// SwiGLU of two bf16 words: gate (g.lo, g.hi) and up (u.lo, u.hi) -> the bf16 word
// (h.lo, h.hi), h = silu(g) * u rounded to bf16 (nearest even).
__device__ __forceinline__ uint32_t swiglu_word(uint32_t g, uint32_t u) {
  const float h0 = silu_times(__uint_as_float(g << 16), __uint_as_float(u << 16));
  const float h1 = silu_times(__uint_as_float(g & 0xFFFF0000u), __uint_as_float(u & 0xFFFF0000u));
  const __nv_bfloat162 h = __floats2bfloat162_rn(h0, h1);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint4 swiglu_uint4(const uint4 &g, const uint4 &u) {
  return make_uint4(swiglu_word(g.x, u.x), swiglu_word(g.y, u.y), swiglu_word(g.z, u.z), swiglu_word(g.w, u.w));
}

// (dg, du) of two elements: gate g, up u, upstream gradient dh, on the packed
// f32x2 pipe.  sigma(g) and sigma(-g) come from t = e^(-|g|) as (1 or t) / (1 + t),
// so neither is formed as 1 - sigma (no cancellation for large |g|) and
// e^(-|g|) never overflows.
__device__ __forceinline__ void swiglu_bwd_pair(float2 g, float2 u, float2 dh, float2 &dg, float2 &du) {
  const float2 s = make_float2(__expf(-0.5f * fabsf(g.x)), __expf(-0.5f * fabsf(g.y)));
  const float2 t = __fmul2_rn(s, s);
  const float2 r = make_float2(rcp_approx(1.0f + t.x), rcp_approx(1.0f + t.y));
  const float2 sig = __fmul2_rn(make_float2(g.x >= 0.0f ? 1.0f : t.x, g.y >= 0.0f ? 1.0f : t.y), r);
  const float2 sig_neg = __fmul2_rn(make_float2(g.x >= 0.0f ? t.x : 1.0f, g.y >= 0.0f ? t.y : 1.0f), r);
  du = __fmul2_rn(dh, __fmul2_rn(g, sig));
  dg = __fmul2_rn(__fmul2_rn(dh, u), __fmul2_rn(sig, __ffma2_rn(g, sig_neg, make_float2(1.0f, 1.0f))));
}

// Eight elements (one 16-byte word of g, u and dh each) -> the bf16 words of dg
// and du (nearest even).
__device__ __forceinline__ void swiglu_bwd_uint4(const uint4 &g, const uint4 &u, const uint4 &dh, uint4 &dg,
                                                 uint4 &du) {
  const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w}, hw[4] = {dh.x, dh.y, dh.z, dh.w};
  uint32_t ow_g[4], ow_u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 gf = make_float2(__uint_as_float(gw[i] << 16), __uint_as_float(gw[i] & 0xFFFF0000u));
    const float2 uf = make_float2(__uint_as_float(uw[i] << 16), __uint_as_float(uw[i] & 0xFFFF0000u));
    const float2 hf = make_float2(__uint_as_float(hw[i] << 16), __uint_as_float(hw[i] & 0xFFFF0000u));
    float2 dgf, duf;
    swiglu_bwd_pair(gf, uf, hf, dgf, duf);
    const __nv_bfloat162 bg = __floats2bfloat162_rn(dgf.x, dgf.y);
    const __nv_bfloat162 bu = __floats2bfloat162_rn(duf.x, duf.y);
    ow_g[i] = *reinterpret_cast<const uint32_t *>(&bg);
    ow_u[i] = *reinterpret_cast<const uint32_t *>(&bu);
  }
  dg = make_uint4(ow_g[0], ow_g[1], ow_g[2], ow_g[3]);
  du = make_uint4(ow_u[0], ow_u[1], ow_u[2], ow_u[3]);
}

}  // namespace fme
