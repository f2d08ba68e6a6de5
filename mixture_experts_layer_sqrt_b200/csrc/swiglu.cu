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
// Streams: forward 3, backward 6 elements moved per hidden element.  The
// arithmetic (one exponential, one division) stays under the copy time for
// bf16.  A warp (or, with few rows, a block of eight) per row, 16-byte loads.
#include "act.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kWarps = 8;  // per block

__device__ __forceinline__ int live_rows_of(int rows, const int32_t *live) {
  if (!live) return rows;
  const int n = *live;
  return n < 0 ? 0 : (n < rows ? n : rows);
}

// SPAN: warps a row (1 or kWarps)
template <typename T, int SPAN>
__global__ void __launch_bounds__(32 * kWarps) swiglu_kernel(int rows, int F, const T *gu, float limit, int mode,
                                                             const int32_t *live, T *h) {
  constexpr int V = Vec16<T>::N;
  const int n_rows = live_rows_of(rows, live);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int RPB = kWarps / SPAN;  // rows a block
  const int part = warp % SPAN;
  for (long r = (long)blockIdx.x * RPB + warp / SPAN; r < n_rows; r += (long)gridDim.x * RPB) {
    const T *g = gu + r * 2 * F, *u = g + F;
#pragma unroll 2
    for (int c = (part * 32 + lane) * V; c < F; c += SPAN * 32 * V) {
      const Vec16<T> gv = load16(g + c), uv = load16(u + c);
      Vec16<T> o;
#pragma unroll
      for (int j = 0; j < V; ++j) o.set(j, swiglu_of(gv.get(j), uv.get(j), limit, mode));
      store16(h + r * F + c, o);
    }
  }
}

template <typename T, int SPAN>
__global__ void __launch_bounds__(32 * kWarps)
    swiglu_backward_kernel(int rows, int F, const T *gu, const T *dh, const float *row_weight, float limit, int mode,
                           const int32_t *live, T *dgu, T *hw, float *drow_weight) {
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
#pragma unroll 2
    for (int c = (part * 32 + lane) * V; c < F; c += SPAN * 32 * V) {
      const Vec16<T> gv = load16(gp + c), uv = load16(up + c), dv = load16(dp + c);
      Vec16<T> og, ou, oh;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float g0 = gv.get(j), u0 = uv.get(j), d = dv.get(j);
        const bool pre = limit > 0.0f && mode == MOE_CLAMP_PREACT;
        const float g = pre ? clip(g0, limit) : g0, u = pre ? clip(u0, limit) : u0;
        const float s = sigmoid_f32(g);
        const float silu = g * s;
        float h = silu * u;
        float dg = d * w * u * (s * (1.0f + g * (1.0f - s))), du = d * w * silu;
        if (pre) {
          if (fabsf(g0) > limit) dg = 0.0f;
          if (fabsf(u0) > limit) du = 0.0f;
        } else if (limit > 0.0f && fabsf(h) > limit) {
          h = clip(h, limit);
          dg = 0.0f;
          du = 0.0f;
        }
        og.set(j, dg);
        ou.set(j, du);
        oh.set(j, w * h);
        sum += d * h;
      }
      store16(dgp + c, og);
      store16(dup + c, ou);
      if (hw) store16(hw + r * F + c, oh);
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

template <typename T>
void forward(int rows, int F, const void *gu, float limit, int mode, const int32_t *live, void *h, int sms,
             cudaStream_t s) {
  const bool sp = spread(rows, sms);
  const int grid = grid_for(rows, sms, sp);
  if (sp) swiglu_kernel<T, kWarps><<<grid, 32 * kWarps, 0, s>>>(rows, F, (const T *)gu, limit, mode, live, (T *)h);
  else swiglu_kernel<T, 1><<<grid, 32 * kWarps, 0, s>>>(rows, F, (const T *)gu, limit, mode, live, (T *)h);
}

template <typename T>
void backward(int rows, int F, const void *gu, const void *dh, const float *rw, float limit, int mode,
              const int32_t *live, void *dgu, void *hw, float *drw, int sms, cudaStream_t s) {
  const bool sp = spread(rows, sms);
  const int grid = grid_for(rows, sms, sp);
  if (sp)
    swiglu_backward_kernel<T, kWarps><<<grid, 32 * kWarps, 0, s>>>(rows, F, (const T *)gu, (const T *)dh, rw, limit,
                                                                   mode, live, (T *)dgu, (T *)hw, drw);
  else
    swiglu_backward_kernel<T, 1><<<grid, 32 * kWarps, 0, s>>>(rows, F, (const T *)gu, (const T *)dh, rw, limit, mode,
                                                              live, (T *)dgu, (T *)hw, drw);
}

}  // namespace

moe_status launch_swiglu(int rows, int F, moe_dtype dtype, const void *gu, float limit, int mode, const int32_t *live,
                         void *h, cudaStream_t s) {
  int sms = 0;
  moe_status st = device_sms(sms);
  if (st != MOE_OK) return st;
  if (dtype == MOE_F32) forward<float>(rows, F, gu, limit, mode, live, h, sms, s);
  else forward<__nv_bfloat16>(rows, F, gu, limit, mode, live, h, sms, s);
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
    backward<float>(rows, F, gu, dh, row_weight, limit, mode, live, dgu, hw, drow_weight, sms, s);
  else
    backward<__nv_bfloat16>(rows, F, gu, dh, row_weight, limit, mode, live, dgu, hw, drow_weight, sms, s);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
