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
// bf16 sources: x / (s rs) is formed as x times (1 + 2^-20) times the rounded
// reciprocal, cut to 18 significant bits.  The product is off by at most 2^-22,
// so a quotient that is exactly one of e2m1's seven ties comes out just above
// it and is cut back onto it; x has 8 bits and s 4, so any other is at least
// 1/256 (relative) away and stays on its side: the codes are those of the exact
// quotient.  blockmax / 6 in the same way (8 bits against e4m3's 5-bit ties).
// fp32 sources divide.
//
// Sources: rows as they lie or through a row map (the dispatch gather done in
// 4 bits), or SwiGLU of gate|up rows, rounded to the rows' type first.  A warp
// per 512 * kHeld elements of a row, up to four: they stay in registers between
// the row maximum and the codes; longer rows are read twice (from L2).  With few
// rows four warps share one whatever its length.
//
// Measured (B200): 49152 rows x 4096 gathered from 8192, with the values, 118 us:
// 513 MB written (a fill of as much takes 131 us), and 77 us without them; 16384 rows
// x 4096 from gate|up 95 us, 108 with the clamp (SwiGLU's accurate exponential and
// reciprocal beside 440 MB).
#include <cuda_fp8.h>

#include "act.cuh"
#include "kernels.h"

namespace moe {

MOE_VIOLATION_COUNTER(violations_quantize)

namespace {

// Warps per block: four rows of one warp each, or one row of SPAN warps.
template <int SPAN>
constexpr int kWarps = SPAN == 1 ? 4 : SPAN;

template <typename T>
struct Group;  // 16 elements of a row
template <>
struct Group<__nv_bfloat16> {
  uint32_t w[8];
  template <bool WIDE>  // 32-byte aligned
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    if constexpr (WIDE) {
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "l"(p));
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
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
  float w[16];
  template <bool WIDE>
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

// Eight codes of t[0..7], element 0 in bits [3:0].
__device__ __forceinline__ uint32_t e2m1x8(const float *t) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}\n"
      : "=r"(r)
      : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
  return r;
}
// 18 significant bits.
__device__ __forceinline__ float cut(float v) { return __uint_as_float(__float_as_uint(v) & ~0x3Fu); }
constexpr float kBump = 1.0f + 9.5367431640625e-07f;  // 1 + 2^-20

struct Out {
  uint8_t *codes, *scales;
  float *row_scale;
  __nv_bfloat16 *values;  // or null
};

// Codes, scale and values (where asked for) of one group with largest magnitude a.
template <typename T, bool WIDE>
__device__ __forceinline__ void emit(const Group<T> &g, float a, float rs, float inv_rs, uint2 *codes, uint8_t *scales,
                                     __nv_bfloat16 *values) {
  const bool bad = !finite(a);
  const float a_rs = a * inv_rs;
  const float s0 = sizeof(T) == 2 ? cut(a_rs * ((1.0f / 6.0f) * kBump)) : __fdiv_rn(a_rs, 6.0f);
  uint32_t s8 = bad ? 0x7Fu : (uint32_t)__nv_cvt_float_to_fp8(s0, __NV_SATFINITE, __NV_E4M3);
  __nv_fp8_e4m3 sc;
  sc.__x = (__nv_fp8_storage_t)s8;
  const float s = (float)sc;
  const float d = s * rs;
  uint32_t q[2];
  float r = 0.0f;
  if (sizeof(T) == 2) {
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    r *= kBump;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = sizeof(T) == 2 ? cut(g.get(8 * i + k) * r) : __fdiv_rn(g.get(8 * i + k), d);
    q[i] = e2m1x8(t);
  }
  if (!(s > 0.0f)) q[0] = q[1] = 0;  // zero or NaN scale
  *codes = make_uint2(q[0], q[1]);
  *scales = (uint8_t)s8;
  if (values) {
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
    if (WIDE) {
      // the values leave L2 first, so that rows gathered again are found there
      // (49152 x 4096 gathered from 8192: 123 -> 119 us, a fill of the outputs 131)
      asm volatile("st.global.L2::evict_first.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(values), "r"(v[0]),
                   "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                   : "memory");
    } else {
      reinterpret_cast<uint4 *>(values)[0] = make_uint4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<uint4 *>(values)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
  }
}

constexpr int kRows = 3;  // a source of rows; 0..2: gate|up with that clamp

// Groups that a lane holds.  bf16, 8192 x 4096 gathered six times / 16384 x 4096
// from gate|up: 8 groups 123 / 135 us, 4 groups 133 / 107, 2 groups 130 / 94:
// copying rows wants the fewest instructions, the exponentials more warps.
template <typename T, int SRC>
constexpr int kHeld = (SRC == kRows ? 8 : 2) * 2 / (int)sizeof(T);

// WIDE: rows and values
// are 32-byte aligned, moved 32 bytes a lane.
template <typename T, int SRC, bool WIDE, int SPAN>
__global__ void __launch_bounds__(32 * kWarps<SPAN>)
    quantize_kernel(int rows, int cols, const T *__restrict__ src, int src_rows, const int32_t *__restrict__ row_token,
                    const int32_t *live, float limit, Out o) {
  constexpr int G = kHeld<T, SRC>;
  constexpr bool SWIGLU = SRC != kRows;
  int n_rows = rows;
  if (live) n_rows = *live < 0 ? 0 : (*live < rows ? *live : rows);
  // SPAN warps a row: warp `part` of them holds every SPAN-th run of 32 groups
  __shared__ float part_max[2][SPAN];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = warp % SPAN;
  const int groups = cols / 16;
  const int chunks = (groups + 32 * SPAN * G - 1) / (32 * SPAN * G);
  constexpr int RPB = kWarps<SPAN> / SPAN;  // rows a block
  int turn = 0;
  for (long r = (long)blockIdx.x * RPB + warp / SPAN; r < n_rows; r += (long)gridDim.x * RPB) {
    long at = r;
    if (!SWIGLU && row_token) {
      at = row_token[r];
      if (at < 0 || at >= src_rows) {  // never read: the row stays as it is
        if (kChecked && lane == 0 && part == 0) note_violation();
        continue;
      }
    }
    const T *x = src + at * (SWIGLU ? 2l : 1l) * cols;
    Group<T> g[G];
    float a[G];
    auto load = [&](int chunk) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int c = ((chunk * G + i) * SPAN + part) * 32 + lane;
        if (c < groups) g[i].template load<WIDE>(x + c * 16);
      }
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int c = ((chunk * G + i) * SPAN + part) * 32 + lane;
        a[i] = 0.0f;
        if (c >= groups) continue;
        if (SWIGLU) {
          Group<T> u;
          u.template load<WIDE>(x + cols + c * 16);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            g[i].set_pair(k, swiglu_of<SRC>(g[i].get(2 * k), u.get(2 * k), limit),
                          swiglu_of<SRC>(g[i].get(2 * k + 1), u.get(2 * k + 1), limit));
        }
        a[i] = g[i].amax();
      }
    };
    int e = 0;
    if (o.row_scale) {
      float m = 0.0f;
      for (int ch = 0; ch < chunks; ++ch) {
        load(ch);
#pragma unroll
        for (int i = 0; i < G; ++i)
          if (finite(a[i])) m = fmaxf(m, a[i]);
      }
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      if (SPAN > 1) {  // the row's warps agree (two sets of slots: one barrier a row is enough)
        if (lane == 0) part_max[turn][part] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < SPAN; ++i) m = fmaxf(m, part_max[turn][i]);
        turn ^= 1;
      }
      e = row_exponent(m);
      if (lane == 0 && part == 0) o.row_scale[r] = pow2(e);
    }
    const float rs = pow2(e), inv_rs = pow2(-e);
    for (int ch = 0; ch < chunks; ++ch) {
      if (chunks > 1 || !o.row_scale) load(ch);
      const int c0 = (ch * G * SPAN + part) * 32 + lane;
      uint2 *codes = reinterpret_cast<uint2 *>(o.codes) + r * groups + c0;
      uint8_t *scales = o.scales + r * groups + c0;
      __nv_bfloat16 *values = o.values ? o.values + (r * cols + c0 * 16) : nullptr;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        constexpr int step = 32 * SPAN;
        if (c0 + i * step < groups)
          emit<T, WIDE>(g[i], a[i], rs, inv_rs, codes + i * step, scales + i * step,
                        values ? values + i * step * 16 : nullptr);
      }
    }
  }
}

template <typename T, int SRC, bool WIDE, int SPAN>
void launch_rows(int rows, int cols, const void *src, int src_rows, const int32_t *row_token, const int32_t *live,
                 float limit, const Out &o, int sms, cudaStream_t s) {
  constexpr int RPB = kWarps<SPAN> / SPAN;
  const long want = ((long)rows + RPB - 1) / RPB, most = (long)sms * 32;
  quantize_kernel<T, SRC, WIDE, SPAN><<<(int)(want < most ? want : most), 32 * kWarps<SPAN>, 0, s>>>(
      rows, cols, (const T *)src, src_rows, row_token, live, limit, o);
}

template <typename T, int SRC, bool WIDE>
void launch_span(int rows, int cols, const void *src, int src_rows, const int32_t *row_token, const int32_t *live,
                 float limit, const Out &o, int sms, cudaStream_t s) {
  constexpr int held = 32 * 16 * kHeld<T, SRC>;  // elements a warp
  if (rows < sms * 4 || cols > 2 * held)
    launch_rows<T, SRC, WIDE, 4>(rows, cols, src, src_rows, row_token, live, limit, o, sms, s);
  else if (cols > held)
    launch_rows<T, SRC, WIDE, 2>(rows, cols, src, src_rows, row_token, live, limit, o, sms, s);
  else
    launch_rows<T, SRC, WIDE, 1>(rows, cols, src, src_rows, row_token, live, limit, o, sms, s);
}

template <typename T, int SRC>
void launch_one(int rows, int cols, const void *src, int src_rows, const int32_t *row_token, const int32_t *live,
                float limit, const Out &o, int sms, cudaStream_t s) {
  // rows are a multiple of 32 bytes; the base addresses may be 16-byte aligned only
  const bool wide = (((uintptr_t)src | (uintptr_t)o.values) & 31u) == 0;
  if (wide) launch_span<T, SRC, true>(rows, cols, src, src_rows, row_token, live, limit, o, sms, s);
  else launch_span<T, SRC, false>(rows, cols, src, src_rows, row_token, live, limit, o, sms, s);
}

template <typename T>
void launch_type(int rows, int cols, bool swiglu, const void *src, int src_rows, const int32_t *row_token,
                 const int32_t *live, float limit, int mode, const Out &o, int sms, cudaStream_t s) {
  const int kind = swiglu ? clamp_kind(limit, mode) : kRows;
  switch (kind) {
    case kNoClamp: launch_one<T, kNoClamp>(rows, cols, src, src_rows, row_token, live, limit, o, sms, s); break;
    case kClampPre: launch_one<T, kClampPre>(rows, cols, src, src_rows, row_token, live, limit, o, sms, s); break;
    case kClampOut: launch_one<T, kClampOut>(rows, cols, src, src_rows, row_token, live, limit, o, sms, s); break;
    default: launch_one<T, kRows>(rows, cols, src, src_rows, row_token, live, limit, o, sms, s); break;
  }
}

}  // namespace

moe_status launch_quantize_nvfp4(int rows, int cols, moe_dtype dtype, bool swiglu, const void *src, int src_rows,
                                 const int32_t *row_token, const int32_t *live, float limit, int mode, void *codes,
                                 void *scales, float *row_scale, void *values, cudaStream_t s) {
  int dev = 0, sms = 148;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  const Out o = {(uint8_t *)codes, (uint8_t *)scales, row_scale, (__nv_bfloat16 *)values};
  if (dtype == MOE_F32)
    launch_type<float>(rows, cols, swiglu, src, src_rows, row_token, live, limit, mode, o, sms, s);
  else
    launch_type<__nv_bfloat16>(rows, cols, swiglu, src, src_rows, row_token, live, limit, mode, o, sms, s);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
