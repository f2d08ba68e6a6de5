// SwiGLU arithmetic shared by swiglu.cu and quantize.cu (internal).
//
// Here a NaN stays a NaN through the clamp; the fused GEMM epilogues' clamp
// (swiglu_h in common.cuh) replaces it by a bound.
#pragma once

#include "common.cuh"

namespace moe {

__device__ __forceinline__ float clip(float v, float limit) { return v < -limit ? -limit : (v > limit ? limit : v); }

__device__ __forceinline__ float sigmoid_f32(float g) { return __fdiv_rn(1.0f, 1.0f + expf(-g)); }

// h = SiLU(clip g) * clip u (limit <= 0: no clip), or the product clipped.
__device__ __forceinline__ float swiglu_of(float g, float u, float limit, int clamp_mode) {
  if (limit > 0.0f && clamp_mode == MOE_CLAMP_PREACT) {
    g = clip(g, limit);
    u = clip(u, limit);
  }
  float h = g * sigmoid_f32(g) * u;
  if (limit > 0.0f && clamp_mode == MOE_CLAMP_OUTPUT) h = clip(h, limit);
  return h;
}

}  // namespace moe
