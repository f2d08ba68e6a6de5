// NVFP4 quantisation of rows: e2m1 codes, an e4m3 scale per 16 elements and,
// on request, a power-of-two fp32 scale per row.
//
//   rs = 1, or 2^ceil(log2(rowmax / 2688))        (2688 = 448 * 6, at least 2^-110)
//   s  = e4m3_rne(blockmax / (6 rs)),  saturating at 448
//   q  = e2m1_rne(x / (s rs)),         saturating at 6;   0 where s = 0
//   value = q * s * rs
//
// The row scale keeps the block scales in e4m3's normal range whatever the
// row's magnitude; a power of two makes every step but the two roundings
// exact, and e4m3's relative step does not depend on it.  A block that holds
// an infinity or a NaN gets the NaN scale (0x7f), takes no part in the row's
// scale and has codes 0: the failure stays visible.
//
// bf16 sources: x / (s rs) is formed as x times the rounded reciprocal and
// then rounded to 18 significant bits.  x has 8 bits and s 4, so a quotient
// that is not exactly on one of e2m1's seven ties is at least 1/256 (relative)
// away from it, and one that is on it is restored by that rounding: the codes
// are those of the exact quotient.  fp32 sources divide.
//
// Sources: rows as they lie or through a row map (the dispatch gather done in
// 4 bits), or SwiGLU of gate|up rows, rounded to the rows' type first.  A warp
// per row; a row of up to 32 * 16 * G elements stays in registers between the
// row maximum and the codes, longer rows are read twice (from L2).
#include <cuda_fp8.h>

#include "act.cuh"
#include "kernels.h"

namespace moe {

MOE_VIOLATION_COUNTER(violations_quantize)

namespace {

constexpr int kWarps = 4;  // per block

template <typename T>
struct Group;  // 16 elements of a row
template <>
struct Group<__nv_bfloat16> {
  static constexpr int kHeld = 8;  // groups a lane holds
  uint32_t w[8];
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
  }
  __device__ __forceinline__ void set_pair(int i, float a, float b) {
    const __nv_bfloat162 o = __floats2bfloat162_rn(a, b);
    w[i] = *reinterpret_cast<const uint32_t *>(&o);
  }
  // largest magnitude; infinity or NaN if one is there (magnitudes compare as integers)
  __device__ __forceinline__ float amax() const {
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    m = (m >> 16) > (m & 0xFFFFu) ? m >> 16 : m & 0xFFFFu;
    return __uint_as_float(m << 16);
  }
};
template <>
struct Group<float> {
  static constexpr int kHeld = 4;
  float w[16];
  __device__ __forceinline__ void load(const float *p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = reinterpret_cast<const float4 *>(p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
  __device__ __forceinline__ float get(int i) const { return w[i]; }
  __device__ __forceinline__ void set_pair(int i, float a, float b) {
    w[2 * i] = a;
    w[2 * i + 1] = b;
  }
  __device__ __forceinline__ float amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(w[i]) & 0x7FFFFFFFu);
    return __uint_as_float(m);
  }
};

__device__ __forceinline__ bool finite(float a) { return a <= 3.4028234664e38f; }

// Exponent of the row scale: ceil(log2(a / 2688)), 2688 = 1.3125 * 2^11.
__device__ __forceinline__ int row_exponent(float a) {
  if (!(a > 0.0f)) return 0;
  const uint32_t b = __float_as_uint(a);
  const int e = (int)(b >> 23) - 127 - 11 + ((b & 0x7FFFFFu) > 0x280000u ? 1 : 0);
  return e < -110 ? -110 : e;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two codes, `lo` in bits [3:0].
__device__ __forceinline__ uint32_t e2m1_pair(float hi, float lo) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "cvt.u32.u8 %0, b;\n\t}\n"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

struct Out {
  uint8_t *codes, *scales;
  float *row_scale;
  __nv_bfloat16 *values;  // or null
};

// Codes, scale and values of one group; rs = 2^e.
template <typename T>
__device__ __forceinline__ void emit(const Group<T> &g, int e, long row, int cols, int group, const Out &o) {
  const float a = g.amax();
  const bool bad = !finite(a);
  const float s0 = __fdiv_rn(a * pow2(-e), 6.0f);
  uint32_t s8 = bad ? 0x7Fu : (uint32_t)__nv_cvt_float_to_fp8(s0, __NV_SATFINITE, __NV_E4M3);
  __nv_fp8_e4m3 sc;
  sc.__x = (__nv_fp8_storage_t)s8;
  const float s = (float)sc;
  const float d = s * pow2(e);
  const bool live = s > 0.0f;  // false for the NaN scale too
  uint32_t q[2] = {0, 0};
  if constexpr (sizeof(T) == 2) {
    const float r = live ? __frcp_rn(d) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float t[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float x = live ? g.get(2 * i + k) : 0.0f;
        t[k] = __uint_as_float((__float_as_uint(x * r) + 0x20u) & ~0x3Fu);
      }
      q[i >> 2] |= e2m1_pair(t[1], t[0]) << (8 * (i & 3));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float t[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) t[k] = live ? __fdiv_rn(g.get(2 * i + k), d) : 0.0f;
      q[i >> 2] |= e2m1_pair(t[1], t[0]) << (8 * (i & 3));
    }
  }
  const long at = row * (cols / 16) + group;
  reinterpret_cast<uint2 *>(o.codes)[at] = make_uint2(q[0], q[1]);
  o.scales[at] = (uint8_t)s8;
  if (o.values) {
    uint32_t v[8];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t h[4];
      asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
          "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
          "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
          "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
          "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
          "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
          : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
          : "r"(q[w]));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * d, f.y * d);
        v[4 * w + j] = *reinterpret_cast<const uint32_t *>(&b);
      }
    }
    uint4 *dst = reinterpret_cast<uint4 *>(o.values + (row * cols + group * 16));
    dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
    dst[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

template <typename T, bool SWIGLU>
__global__ void __launch_bounds__(32 * kWarps)
    quantize_kernel(int rows, int cols, const T *src, int src_rows, const int32_t *row_token, const int32_t *live,
                    float limit, int mode, Out o) {
  constexpr int G = Group<T>::kHeld;
  int n_rows = rows;
  if (live) n_rows = *live < 0 ? 0 : (*live < rows ? *live : rows);
  const int lane = threadIdx.x & 31;
  const int groups = cols / 16;
  const int chunks = (groups + 32 * G - 1) / (32 * G);
  const long stride = (long)gridDim.x * kWarps;
  for (long r = (long)blockIdx.x * kWarps + (threadIdx.x >> 5); r < n_rows; r += stride) {
    long at = r;
    if (!SWIGLU && row_token) {
      at = row_token[r];
      if (at < 0 || at >= src_rows) {  // never read: the row stays as it is
        if (kChecked && lane == 0) note_violation();
        continue;
      }
    }
    const T *x = src + at * (SWIGLU ? 2l : 1l) * cols;
    Group<T> g[G];
    auto load = [&](int chunk) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int c = (chunk * G + i) * 32 + lane;
        if (c >= groups) continue;
        g[i].load(x + c * 16);
        if (SWIGLU) {
          Group<T> u;
          u.load(x + cols + c * 16);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            g[i].set_pair(k, swiglu_of(g[i].get(2 * k), u.get(2 * k), limit, mode),
                          swiglu_of(g[i].get(2 * k + 1), u.get(2 * k + 1), limit, mode));
        }
      }
    };
    int e = 0;
    if (o.row_scale) {
      float m = 0.0f;
      for (int ch = 0; ch < chunks; ++ch) {
        load(ch);
#pragma unroll
        for (int i = 0; i < G; ++i) {
          if ((ch * G + i) * 32 + lane >= groups) continue;
          const float a = g[i].amax();
          if (finite(a)) m = fmaxf(m, a);
        }
      }
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      e = row_exponent(m);
      if (lane == 0) o.row_scale[r] = pow2(e);
    }
    for (int ch = 0; ch < chunks; ++ch) {
      if (chunks > 1 || !o.row_scale) load(ch);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int c = (ch * G + i) * 32 + lane;
        if (c < groups) emit(g[i], e, r, cols, c, o);
      }
    }
  }
}

template <typename T, bool SWIGLU>
void launch_one(int rows, int cols, const void *src, int src_rows, const int32_t *row_token, const int32_t *live,
                float limit, int mode, const Out &o, int sms, cudaStream_t s) {
  const long want = ((long)rows + kWarps - 1) / kWarps;
  const int grid = (int)(want < (long)sms * 16 ? want : (long)sms * 16);
  quantize_kernel<T, SWIGLU><<<grid, 32 * kWarps, 0, s>>>(rows, cols, (const T *)src, src_rows, row_token, live, limit,
                                                          mode, o);
}

}  // namespace

moe_status launch_quantize_nvfp4(int rows, int cols, moe_dtype dtype, bool swiglu, const void *src, int src_rows,
                                 const int32_t *row_token, const int32_t *live, float limit, int mode, void *codes,
                                 void *scales, float *row_scale, void *values, cudaStream_t s) {
  int dev = 0, sms = 148;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  const Out o = {(uint8_t *)codes, (uint8_t *)scales, row_scale, (__nv_bfloat16 *)values};
  if (dtype == MOE_F32) {
    if (swiglu) launch_one<float, true>(rows, cols, src, src_rows, row_token, live, limit, mode, o, sms, s);
    else launch_one<float, false>(rows, cols, src, src_rows, row_token, live, limit, mode, o, sms, s);
  } else {
    if (swiglu) launch_one<__nv_bfloat16, true>(rows, cols, src, src_rows, row_token, live, limit, mode, o, sms, s);
    else launch_one<__nv_bfloat16, false>(rows, cols, src, src_rows, row_token, live, limit, mode, o, sms, s);
  }
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
