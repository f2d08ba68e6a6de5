// SwiGLU on stored gate|up rows, and its gradient with the routing weights.
//
//   gu[r] = (g, u), 2 F columns;  h = SiLU(g) u,  SiLU(g) = g s,  s = 1 / (1 + e^-g)
//
// The layer's product behind h is y[r] = w_r (h[r] W_down^T).  From
// d[r] = dy[r] W_down, the gradient of the unweighted product's input:
//   dg = w d u s (1 + g (1 - s)),   du = w d g s      (gradient of gate|up)
//   hw = w h                                          (dW_down = dy^T hw)
//   dw_r = sum_f d h                                  (gradient of the routing weight)
// all from one reading of gu and d, nothing kept from the forward pass but gu.
// With the clamp at L, a clipped g or u (|v| > L) gets no gradient; in the
// output mode h is clipped and a clipped h passes none.
//
// Streams: forward 3, backward 6 elements moved per hidden element.  A warp (or,
// with few rows, a block of eight) per row, 16-byte loads, the next piece loaded
// ahead.  Measured (B200, bf16): backward 65536 x 1536 206 us = 5.87 TB/s (a copy:
// 6.5; with the correctly rounded reciprocal as well it took 243 us);
// forward 16384 x 4096 75 us = 5.3 TB/s.
#include "act.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kWarps = 8;  // per block

// 16 bytes of T from fp32 values, each rounded once.
template <typename T>
__device__ __forceinline__ Vec16<T> pack16(const float *f);
template <>
__device__ __forceinline__ Vec16<float> pack16<float>(const float *f) {
  Vec16<float> r;
  r.v = make_float4(f[0], f[1], f[2], f[3]);
  return r;
}
template <>
__device__ __forceinline__ Vec16<__nv_bfloat16> pack16<__nv_bfloat16>(const float *f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&p);
  }
  Vec16<__nv_bfloat16> r;
  r.v = make_uint4(w[0], w[1], w[2], w[3]);
  return r;
}

__device__ __forceinline__ int live_rows_of(int rows, const int32_t *live) {
  if (!live) return rows;
  const int n = *live;
  return n < 0 ? 0 : (n < rows ? n : rows);
}

// SPAN: warps a row (1 or kWarps)
template <typename T, int SPAN, int CLAMP>
__global__ void __launch_bounds__(32 * kWarps) swiglu_kernel(int rows, int F, const T *__restrict__ gu, float limit,
                                                             const int32_t *live, T *__restrict__ h) {
  constexpr int V = Vec16<T>::N;
  const int n_rows = live_rows_of(rows, live);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int RPB = kWarps / SPAN;  // rows a block
  const int part = warp % SPAN;
  for (long r = (long)blockIdx.x * RPB + warp / SPAN; r < n_rows; r += (long)gridDim.x * RPB) {
    const T *g = gu + r * 2 * F, *u = g + F;
    constexpr int step = SPAN * 32 * V;
    int c = (part * 32 + lane) * V;
    Vec16<T> gn, un;  // the next piece, loaded ahead
    if (c < F) gn = load16(g + c), un = load16(u + c);
#pragma unroll 2
    for (; c < F; c += step) {
      const Vec16<T> gv = gn, uv = un;
      if (c + step < F) gn = load16(g + c + step), un = load16(u + c + step);
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = swiglu_of<CLAMP>(gv.get(j), uv.get(j), limit);
      store16(h + r * F + c, pack16<T>(o));
    }
  }
}

template <typename T, int SPAN, int CLAMP>
__global__ void __launch_bounds__(32 * kWarps)
    swiglu_backward_kernel(int rows, int F, const T *gu, const T *__restrict__ dh, const float *__restrict__ row_weight,
                           float limit, const int32_t *live, T *dgu, T *__restrict__ hw, float *drow_weight) {
  constexpr int V = Vec16<T>::N;
  __shared__ float part_sum[kWarps];
  const int n_rows = live_rows_of(rows, live);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int RPB = kWarps / SPAN;
  const int part = warp % SPAN;
  for (long r = (long)blockIdx.x * RPB + warp / SPAN; r < n_rows; r += (long)gridDim.x * RPB) {
    const T *gp = gu + r * 2 * F, *up = gp + F, *dp = dh + r * F;
    T *dgp = dgu + r * 2 * F, *dup = dgp + F;
    const float w = row_weight ? row_weight[r] : 1.0f;
    float sum = 0.0f;
    constexpr int step = SPAN * 32 * V;
    int c = (part * 32 + lane) * V;
    Vec16<T> gn, un, dn;  // the next piece, loaded ahead
    if (c < F) gn = load16(gp + c), un = load16(up + c), dn = load16(dp + c);
#pragma unroll 1
    for (; c < F; c += step) {
      const Vec16<T> gv = gn, uv = un, dv = dn;
      if (c + step < F) gn = load16(gp + c + step), un = load16(up + c + step), dn = load16(dp + c + step);
      float og[V], ou[V], oh[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float g0 = gv.get(j), u0 = uv.get(j), d = dv.get(j);
        const float g = CLAMP == kClampPre ? clip(g0, limit) : g0, u = CLAMP == kClampPre ? clip(u0, limit) : u0;
        const float s = sizeof(T) == 2 ? sigmoid_fast(g) : sigmoid_f32(g);
        const float silu = g * s, dw = d * w;
        float h = silu * u;
        og[j] = dw * u * fmaf(silu, 1.0f - s, s);
        ou[j] = dw * silu;
        if (CLAMP == kClampPre) {
          if (fabsf(g0) > limit) og[j] = 0.0f;
          if (fabsf(u0) > limit) ou[j] = 0.0f;
        } else if (CLAMP == kClampOut) {
          if (fabsf(h) > limit) {
            og[j] = 0.0f;
            ou[j] = 0.0f;
          }
          h = clip(h, limit);
        }
        oh[j] = w * h;
        sum = fmaf(d, h, sum);
      }
      store16(dgp + c, pack16<T>(og));
      store16(dup + c, pack16<T>(ou));
      if (hw) store16(hw + r * F + c, pack16<T>(oh));
    }
    if (drow_weight) {
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (SPAN == 1) {
        if (lane == 0) drow_weight[r] = sum;
      } else {
        if (lane == 0) part_sum[warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
          float all = 0.0f;
          for (int i = 0; i < kWarps; ++i) all += part_sum[i];
          drow_weight[r] = all;
        }
        __syncthreads();
      }
    }
  }
}

moe_status device_sms(int &sms) {
  int dev = 0;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  return MOE_OK;
}

// Blocks that share a row are used while a warp a row would leave the GPU
// with less than one block an SM.
inline bool spread(int rows, int sms) { return rows < sms * kWarps; }
inline int grid_for(int rows, int sms, bool spread_rows) {
  const long blocks = spread_rows ? rows : ((long)rows + kWarps - 1) / kWarps;
  return (int)(blocks < (long)sms * 8 ? blocks : (long)sms * 8);
}

template <typename T, int CLAMP>
void forward(int rows, int F, const void *gu, float limit, const int32_t *live, void *h, int sms, cudaStream_t s) {
  const bool sp = spread(rows, sms);
  const int grid = grid_for(rows, sms, sp);
  if (sp) swiglu_kernel<T, kWarps, CLAMP><<<grid, 32 * kWarps, 0, s>>>(rows, F, (const T *)gu, limit, live, (T *)h);
  else swiglu_kernel<T, 1, CLAMP><<<grid, 32 * kWarps, 0, s>>>(rows, F, (const T *)gu, limit, live, (T *)h);
}

template <typename T, int CLAMP>
void backward(int rows, int F, const void *gu, const void *dh, const float *rw, float limit, const int32_t *live,
              void *dgu, void *hw, float *drw, int sms, cudaStream_t s) {
  const bool sp = spread(rows, sms);
  const int grid = grid_for(rows, sms, sp);
  if (sp)
    swiglu_backward_kernel<T, kWarps, CLAMP><<<grid, 32 * kWarps, 0, s>>>(rows, F, (const T *)gu, (const T *)dh, rw,
                                                                          limit, live, (T *)dgu, (T *)hw, drw);
  else
    swiglu_backward_kernel<T, 1, CLAMP><<<grid, 32 * kWarps, 0, s>>>(rows, F, (const T *)gu, (const T *)dh, rw, limit,
                                                                     live, (T *)dgu, (T *)hw, drw);
}

// f<T, CLAMP>(args...) for the element type and clamp of the call
#define MOE_BY_CLAMP(f, T, ...)                                          \
  do {                                                                   \
    switch (clamp_kind(limit, mode)) {                                   \
      case kNoClamp: f<T, kNoClamp>(__VA_ARGS__); break;                 \
      case kClampPre: f<T, kClampPre>(__VA_ARGS__); break;               \
      default: f<T, kClampOut>(__VA_ARGS__); break;                      \
    }                                                                    \
  } while (0)

}  // namespace

moe_status launch_swiglu(int rows, int F, moe_dtype dtype, const void *gu, float limit, int mode, const int32_t *live,
                         void *h, cudaStream_t s) {
  int sms = 0;
  moe_status st = device_sms(sms);
  if (st != MOE_OK) return st;
  if (dtype == MOE_F32) MOE_BY_CLAMP(forward, float, rows, F, gu, limit, live, h, sms, s);
  else MOE_BY_CLAMP(forward, __nv_bfloat16, rows, F, gu, limit, live, h, sms, s);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

moe_status launch_swiglu_backward(int rows, int F, moe_dtype dtype, const void *gu, const void *dh,
                                  const float *row_weight, float limit, int mode, const int32_t *live, void *dgu,
                                  void *hw, float *drow_weight, cudaStream_t s) {
  int sms = 0;
  moe_status st = device_sms(sms);
  if (st != MOE_OK) return st;
  if (dtype == MOE_F32)
    MOE_BY_CLAMP(backward, float, rows, F, gu, dh, row_weight, limit, live, dgu, hw, drow_weight, sms, s);
  else
    MOE_BY_CLAMP(backward, __nv_bfloat16, rows, F, gu, dh, row_weight, limit, live, dgu, hw, drow_weight, sms, s);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
