// C ABI of the products grouped by expert, NVFP4 quantisation and SwiGLU:
// argument checks, then the kernels.
#include <limits.h>

#include "common.cuh"
#include "kernels.h"
#include "tma_host.h"

namespace moe {
namespace {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool ok_ptr(const void *p) { return p != nullptr && aligned16(p); }
inline bool ok_opt4(const void *p) { return ((uintptr_t)p & 3u) == 0; }  // optional float or int32 arrays

moe_status validate(const MoEGrouped *g) {
  if (!g || g->groups < 1 || g->rows < 0 || g->n <= 0 || g->k <= 0) return MOE_ERR_INVALID_ARG;
  if (g->dtype != MOE_F32 && g->dtype != MOE_BF16 && g->dtype != MOE_NVFP4) return MOE_ERR_INVALID_ARG;
  if (g->out_dtype != MOE_F32 && g->out_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (g->dtype == MOE_F32 && g->out_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (g->groups > 1024) return MOE_ERR_UNSUPPORTED;
  if (g->n % 8 || g->k % (g->dtype == MOE_NVFP4 ? 32 : 8)) return MOE_ERR_UNSUPPORTED;  // 16-byte rows
  // scale rows of other lengths are addressed by 32-bit offsets within a tile (gemm_grouped_fp4.cu)
  if (g->dtype == MOE_NVFP4 && g->k % 256 && g->k > 1 << 26) return MOE_ERR_UNSUPPORTED;
  if (g->rows > INT_MAX / 2 || g->n > INT_MAX / 2 || g->k > INT_MAX / 2) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// What the products check alike, in this order: sizes, workspace, offsets.
moe_status check_call(const MoEGrouped *g, bool nvfp4, const int32_t *offsets, void *ws, size_t ws_bytes) {
  moe_status st = validate(g);
  if (st != MOE_OK) return st;
  if ((g->dtype == MOE_NVFP4) != nvfp4 || !ws || !ok_opt4(ws)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < kStatusBytes) return MOE_ERR_WORKSPACE;
  if ((!offsets && g->groups != 1) || !ok_opt4(offsets)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_rows(int rows, int cols, int multiple, moe_dtype dtype, const int32_t *live) {
  if (rows < 0 || cols <= 0 || !ok_opt4(live)) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (cols % multiple || cols > INT_MAX / 4 || rows > INT_MAX / 2) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
inline bool ok_clamp(float clamp, moe_clamp_mode mode) {
  return clamp >= 0.0f && (mode == MOE_CLAMP_PREACT || mode == MOE_CLAMP_OUTPUT);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grouped_workspace_size(const MoEGrouped *g) { return validate(g) == MOE_OK ? kStatusBytes : 0; }

moe_status moe_grouped_matmul(const MoEGrouped *g, const void *a, const int32_t *expert_offsets, const void *w,
                              int transposed, const float *row_weight, void *y, void *ws, size_t ws_bytes,
                              moe_stream_t stream) {
  moe_status st = check_call(g, false, expert_offsets, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (g->rows == 0) return MOE_OK;
  if (!ok_ptr(a) || !ok_ptr(w) || !ok_ptr(y) || !ok_opt4(row_weight)) return MOE_ERR_INVALID_ARG;
  if (g->dtype == MOE_F32)
    return launch_grouped_f32(*g, a, expert_offsets, w, transposed != 0, row_weight, y, (cudaStream_t)stream);
  if (!tma_encode_fn()) return MOE_ERR_CUDA;
  return launch_grouped_bf16(*g, a, expert_offsets, w, transposed != 0, row_weight, y, (int *)ws,
                             (cudaStream_t)stream);
}

moe_status moe_grouped_wgrad(const MoEGrouped *g, const void *dy, const void *a, const int32_t *expert_offsets,
                             int accumulate, void *dw, void *ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status st = check_call(g, false, expert_offsets, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (!ok_ptr(dw)) return MOE_ERR_INVALID_ARG;
  if (g->rows == 0) {  // every group is empty
    if (accumulate) return MOE_OK;
    const size_t bytes = (size_t)g->groups * g->n * g->k * (g->out_dtype == MOE_F32 ? 4 : 2);
    MOE_CUDA_TRY(cudaMemsetAsync(dw, 0, bytes, (cudaStream_t)stream));
    return MOE_OK;
  }
  if (!ok_ptr(dy) || !ok_ptr(a)) return MOE_ERR_INVALID_ARG;
  if (g->dtype == MOE_F32)
    return launch_grouped_wgrad_f32(*g, dy, a, expert_offsets, accumulate != 0, dw, (cudaStream_t)stream);
  if (!tma_encode_fn()) return MOE_ERR_CUDA;
  return launch_grouped_wgrad_bf16(*g, dy, a, expert_offsets, accumulate != 0, dw, (int *)ws, (cudaStream_t)stream);
}

moe_status moe_grouped_matmul_nvfp4(const MoEGrouped *g, const void *a, const void *a_scales, const float *a_row_scale,
                                    const int32_t *expert_offsets, const void *w, const void *w_scales,
                                    const float *w_row_scale, const float *row_weight, void *y, void *ws,
                                    size_t ws_bytes, moe_stream_t stream) {
  moe_status st = check_call(g, true, expert_offsets, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (g->rows == 0) return MOE_OK;
  if (!ok_ptr(a) || !ok_ptr(a_scales) || !ok_ptr(w) || !ok_ptr(w_scales) || !ok_ptr(y)) return MOE_ERR_INVALID_ARG;
  if (!ok_opt4(a_row_scale) || !ok_opt4(w_row_scale) || !ok_opt4(row_weight)) return MOE_ERR_INVALID_ARG;
  if (!tma_encode_fn()) return MOE_ERR_CUDA;
  return launch_grouped_nvfp4(*g, a, a_scales, a_row_scale, expert_offsets, w, w_scales, w_row_scale, row_weight, y,
                              (int *)ws, (cudaStream_t)stream);
}

moe_status moe_quantize_nvfp4(int rows, int cols, moe_dtype dtype, const void *x, int x_rows, const int32_t *row_token,
                              const int32_t *live_rows, void *codes, void *scales, float *row_scale, void *values,
                              moe_stream_t stream) {
  moe_status st = check_rows(rows, cols, 16, dtype, live_rows);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  if (x_rows <= 0 || (!row_token && x_rows < rows)) return MOE_ERR_INVALID_ARG;
  if (!ok_ptr(x) || !ok_ptr(codes) || !scales || !aligned16(values)) return MOE_ERR_INVALID_ARG;
  if (!ok_opt4(row_token) || !ok_opt4(row_scale)) return MOE_ERR_INVALID_ARG;
  return launch_quantize_nvfp4(rows, cols, dtype, false, x, x_rows, row_token, live_rows, 0.0f, 0, codes, scales,
                               row_scale, values, (cudaStream_t)stream);
}

moe_status moe_swiglu_quantize_nvfp4(int rows, int cols, moe_dtype dtype, const void *gu, float clamp,
                                     moe_clamp_mode clamp_mode, const int32_t *live_rows, void *codes, void *scales,
                                     float *row_scale, void *values, moe_stream_t stream) {
  moe_status st = check_rows(rows, cols, 16, dtype, live_rows);
  if (st != MOE_OK) return st;
  if (!ok_clamp(clamp, clamp_mode)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!ok_ptr(gu) || !ok_ptr(codes) || !scales || !aligned16(values) || !ok_opt4(row_scale))
    return MOE_ERR_INVALID_ARG;
  return launch_quantize_nvfp4(rows, cols, dtype, true, gu, rows, nullptr, live_rows, clamp, clamp_mode, codes, scales,
                               row_scale, values, (cudaStream_t)stream);
}

moe_status moe_swiglu(int rows, int F, moe_dtype dtype, const void *gu, float clamp, moe_clamp_mode clamp_mode,
                      const int32_t *live_rows, void *h, moe_stream_t stream) {
  moe_status st = check_rows(rows, F, 8, dtype, live_rows);
  if (st != MOE_OK) return st;
  if (!ok_clamp(clamp, clamp_mode)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!ok_ptr(gu) || !ok_ptr(h)) return MOE_ERR_INVALID_ARG;
  return launch_swiglu(rows, F, dtype, gu, clamp, clamp_mode, live_rows, h, (cudaStream_t)stream);
}

moe_status moe_swiglu_backward(int rows, int F, moe_dtype dtype, const void *gu, const void *dh,
                               const float *row_weight, float clamp, moe_clamp_mode clamp_mode,
                               const int32_t *live_rows, void *dgu, void *hw, float *drow_weight, moe_stream_t stream) {
  moe_status st = check_rows(rows, F, 8, dtype, live_rows);
  if (st != MOE_OK) return st;
  if (!ok_clamp(clamp, clamp_mode)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!ok_ptr(gu) || !ok_ptr(dh) || !ok_ptr(dgu) || !aligned16(hw)) return MOE_ERR_INVALID_ARG;
  if (!ok_opt4(row_weight) || !ok_opt4(drow_weight)) return MOE_ERR_INVALID_ARG;
  return launch_swiglu_backward(rows, F, dtype, gu, dh, row_weight, clamp, clamp_mode, live_rows, dgu, hw, drow_weight,
                                (cudaStream_t)stream);
}

}  // extern "C"
