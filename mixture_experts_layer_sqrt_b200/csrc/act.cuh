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

// For bf16 gradients: the hardware's exponential and reciprocal, within 2^-20 of
// the value for |g| < 10, against the 2^-8 of the store (27 instead of 56
// instructions an element, the backward pass 69 -> 54 us at 16384 x 1536).
__device__ __forceinline__ float sigmoid_fast(float g) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-g)));
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
