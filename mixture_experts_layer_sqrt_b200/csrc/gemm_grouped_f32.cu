// Products grouped by expert and their gradients in fp32 on CUDA cores (the
// tensor cores' TF32 cannot meet fp32's error); see gemm_grouped.cu for the
// three modes.  64 x 64 outputs per block of 256 threads, 4 x 4 per thread,
// reduction in steps of 16 through shared memory with the next step's loads in
// flight; fp32 FMA in the reduction's order, no split of a sum.
#include "grouped.cuh"
#include "kernels.h"

namespace moe {

MOE_VIOLATION_COUNTER(violations_gemm_grouped_f32)

namespace {

using namespace grouped;

enum Mode { NT = 0, NN = 1, TN = 2 };
constexpr int BM = 64, BN = 64, BK = 16;

// Four consecutive elements starting at (row, col) of a row-major matrix with
// `ld` columns; zeros at row >= rows or col >= ld (ld is a multiple of 4).
__device__ __forceinline__ float4 load4(const float *m, long row, int col, long rows, int ld) {
  if (row >= rows || col >= ld) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  return __ldg(reinterpret_cast<const float4 *>(m + row * ld + col));
}

// M side: rows of the group (NT, NN) or features of dy (TN); N side: output columns.
template <Mode MODE>
__global__ void __launch_bounds__(256) grouped_f32(int rows, int N, int K, int E, const int32_t *__restrict__ offsets,
                                                   const float *__restrict__ A, const float *__restrict__ B,
                                                   const float *__restrict__ row_weight, int accumulate, float *out) {
  __shared__ __align__(16) float As[2][BK][BM + 4];
  __shared__ __align__(16) float Bs[2][BK][BN + 4];
  __shared__ int start[MAX_E + 1];

  int e, m0, n0 = blockIdx.y * BN, m_end, red, row0;
  if (MODE == TN) {
    e = blockIdx.z;
    if (kChecked && offsets && (offsets[e] < 0 || offsets[e + 1] < offsets[e])) {
      if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) note_violation();
      return;
    }
    m0 = blockIdx.x * BM;
    m_end = N;
    row0 = seg_begin(offsets, rows, e);
    red = seg_end(offsets, rows, e) - row0;
    if (red <= 0 && accumulate) return;
  } else {
    if (threadIdx.x < 32) {
      const bool ok = scan_tiles(offsets, rows, E, BM, start);
      if (kChecked && !ok && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) note_violation();
    }
    __syncthreads();
    if ((int)blockIdx.x >= start[E]) return;
    e = find_group(start, E, 1, blockIdx.x);
    row0 = seg_begin(offsets, rows, e);
    m0 = row0 + ((int)blockIdx.x - start[e]) * BM;
    m_end = seg_end(offsets, rows, e);
    red = K;
  }
  const float *We = MODE == TN ? nullptr : B + (long)e * N * K;

  // this thread's piece of a stage: 4 elements of each operand
  const int t = threadIdx.x;
  const int kr = t >> 2, kc = (t & 3) * 4;    // K-major operand: row kr, reduction kc..kc+3
  const int mr = t >> 4, mc = (t & 15) * 4;   // MN-major operand: reduction mr, feature mc..mc+3
  float4 ra, rb;
  auto fetch = [&](int k0) {
    if (MODE == TN) {
      ra = load4(A, row0 + k0 + mr, m0 + mc, (long)row0 + red, N);
      rb = load4(B, row0 + k0 + mr, n0 + mc, (long)row0 + red, K);
    } else {
      ra = load4(A, (long)m0 + kr, k0 + kc, m_end, K);
      if (MODE == NT) rb = load4(We, (long)n0 + kr, k0 + kc, N, K);
      else rb = load4(We, (long)k0 + mr, n0 + mc, K, N);
    }
  };
  auto put = [&](int b) {
    if (MODE == TN) {
      *reinterpret_cast<float4 *>(&As[b][mr][mc]) = ra;
    } else {
      As[b][kc][kr] = ra.x;
      As[b][kc + 1][kr] = ra.y;
      As[b][kc + 2][kr] = ra.z;
      As[b][kc + 3][kr] = ra.w;
    }
    if (MODE == NT) {
      Bs[b][kc][kr] = rb.x;
      Bs[b][kc + 1][kr] = rb.y;
      Bs[b][kc + 2][kr] = rb.z;
      Bs[b][kc + 3][kr] = rb.w;
    } else {
      *reinterpret_cast<float4 *>(&Bs[b][mr][mc]) = rb;
    }
  };

  const int tx = t & 15, ty = t >> 4;
  float acc[4][4] = {};
  const int steps = (red + BK - 1) / BK;
  if (steps > 0) {
    fetch(0);
    put(0);
  }
  __syncthreads();
  for (int i = 0; i < steps; ++i) {
    const int b = i & 1;
    if (i + 1 < steps) fetch((i + 1) * BK);
#pragma unroll
    for (int kk = 0; kk < BK; ++kk) {
      const float4 a4 = *reinterpret_cast<const float4 *>(&As[b][kk][ty * 4]);
      const float4 b4 = *reinterpret_cast<const float4 *>(&Bs[b][kk][tx * 4]);
      const float av[4] = {a4.x, a4.y, a4.z, a4.w}, bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[x][y] = fmaf(av[x], bv[y], acc[x][y]);
    }
    if (i + 1 < steps) put(b ^ 1);
    __syncthreads();
  }

  const int ld = MODE == TN ? K : N;
  const int col = n0 + tx * 4;
  if (col >= ld) return;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int r = m0 + ty * 4 + x;
    if (r >= m_end) continue;
    const float w = MODE != TN && row_weight ? row_weight[r] : 1.0f;
    float4 v = make_float4(acc[x][0] * w, acc[x][1] * w, acc[x][2] * w, acc[x][3] * w);
    float4 *dst = reinterpret_cast<float4 *>(out + ((MODE == TN ? (long)e * N : 0l) + r) * ld + col);
    if (MODE == TN && accumulate) {
      const float4 o = *dst;
      v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
    }
    *dst = v;
  }
}

}  // namespace

moe_status launch_grouped_f32(const MoEGrouped &g, const void *a, const int32_t *offsets, const void *w,
                              bool transposed, const float *row_weight, void *y, cudaStream_t s) {
  const long used = g.rows < g.groups ? g.rows : g.groups;
  const long mt = (long)(g.rows + BM - 1) / BM + used;
  const long nt = (g.n + BN - 1) / BN;
  if (mt > 0x7fffffffl || nt > 65535) return MOE_ERR_UNSUPPORTED;
  dim3 grid((unsigned)mt, (unsigned)nt);
  if (transposed)
    grouped_f32<NN><<<grid, 256, 0, s>>>(g.rows, g.n, g.k, g.groups, offsets, (const float *)a, (const float *)w,
                                         row_weight, 0, (float *)y);
  else
    grouped_f32<NT><<<grid, 256, 0, s>>>(g.rows, g.n, g.k, g.groups, offsets, (const float *)a, (const float *)w,
                                         row_weight, 0, (float *)y);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

moe_status launch_grouped_wgrad_f32(const MoEGrouped &g, const void *dy, const void *a, const int32_t *offsets,
                                    bool accumulate, void *dw, cudaStream_t s) {
  const long nt = (g.k + BN - 1) / BN;
  if (nt > 65535) return MOE_ERR_UNSUPPORTED;
  dim3 grid((unsigned)((g.n + BM - 1) / BM), (unsigned)nt, (unsigned)g.groups);
  grouped_f32<TN><<<grid, 256, 0, s>>>(g.rows, g.n, g.k, g.groups, offsets, (const float *)dy, (const float *)a,
                                       nullptr, accumulate, (float *)dw);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
