// SwiGLU arithmetic shared by swiglu.cu and quantize.cu (internal).
//
// Here a NaN stays a NaN through the clamp; the fused GEMM epilogues' clamp
// (swiglu_h in common.cuh) replaces it by a bound.
#pragma once

#include "common.cuh"

namespace moe {

__device__ __forceinline__ float clip(float v, float limit) { return v < -limit ? -limit : (v > limit ? limit : v); }

// IEEE reciprocal and the accurate exponential: the forward value feeds the 4-bit
// rounding, where a changed last bit of h can move a whole code.
__device__ __forceinline__ float sigmoid_f32(float g) { return __frcp_rn(1.0f + expf(-g)); }

// For gradients of bf16 rows: the accurate exponential (2 steps) and the hardware's
// reciprocal (1 step), together within 7 * 2^-24 of the value (0 from g = -87.3 down,
// where it is below fp32's normal range).  The routing weights' gradient is a sum of
// d h in fp32, so the bf16 store of the other outputs is no ground for less: the
// hardware's exponential is off by 2^-18 at g = -55.  Backward pass of 65536 x 1536: 206 us so, 203
// with the hardware's exponential, 243 with both accurate.
__device__ __forceinline__ float sigmoid_fast(float g) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + expf(-g)));
  return r;
}

enum Clamp { kNoClamp = 0, kClampPre = 1, kClampOut = 2 };
inline int clamp_kind(float limit, int mode) {
  return !(limit > 0.0f) ? kNoClamp : mode == MOE_CLAMP_PREACT ? kClampPre : kClampOut;
}

// h = SiLU(clip g) * clip u, or the product clipped.
template <int CLAMP>
__device__ __forceinline__ float swiglu_of(float g, float u, float limit) {
  if (CLAMP == kClampPre) {
    g = clip(g, limit);
    u = clip(u, limit);
  }
  const float h = g * sigmoid_f32(g) * u;
  return CLAMP == kClampOut ? clip(h, limit) : h;
}

}  // namespace moe
