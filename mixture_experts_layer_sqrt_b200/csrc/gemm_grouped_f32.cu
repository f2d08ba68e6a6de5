// Products grouped by expert and their gradients in fp32 on CUDA cores (the
// tensor cores' TF32 cannot meet fp32's error); see gemm_grouped.cu for the
// three modes.  32 x 64 outputs per block of 128 threads, 4 x 4 per thread (a
// group of a small layer has a few dozen rows), reduction in stages of 32
// copied asynchronously two stages ahead: with one stage of registers ahead the
// 64-token layer's gate|up product took 8.0 us, bound by load latency.  A
// thread's sum is one fp32 FMA chain in the reduction's order.
//
// A K-major operand lies as [row][k] (pitch 36): a thread's rows are 8 or 16
// apart, so that a quarter warp's 16-byte reads fall into different banks; an
// MN-major one as [k][feature], a thread's four features side by side.
#include "grouped.cuh"
#include "kernels.h"

namespace moe {

MOE_VIOLATION_COUNTER(violations_gemm_grouped_f32)

namespace {

using namespace grouped;

enum Mode { NT = 0, NN = 1, TN = 2 };
constexpr int BM = 32, BN = 64, BK = 32;
constexpr int kThreads = 128;
constexpr int kStages = 3;
constexpr int kPitch = BK + 4;                  // K-major
constexpr int A_FLOATS = BM * kPitch;           // also holds [BK][BM + 4]
constexpr int B_FLOATS = BN * kPitch;           // also holds [BK][BN + 4]
static_assert(kStages * A_FLOATS >= MAX_E + 1, "the offsets fit before the stages");
static_assert(BK * (BM + 4) <= A_FLOATS && BK * (BN + 4) <= B_FLOATS, "either layout fits");

// 16 bytes to shared memory, zeros when !in (nothing is read then).
__device__ __forceinline__ void copy16(float *dst, const float *src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_addr(dst)), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}

// A tile of R rows (features) x BK reduction elements.  K-major: rows row0.. of
// a matrix with `ld` columns, columns k0..; MN-major: rows k0.., columns row0...
template <int R, bool K_MAJOR>
__device__ __forceinline__ void copy_tile(float *dst, const float *m, long row0, long k0, long rows, long ks, long ld) {
#pragma unroll
  for (int j = 0; j < R * BK / 4 / kThreads; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (K_MAJOR) {
      const int r = i / (BK / 4), c = i % (BK / 4) * 4;
      const bool in = row0 + r < rows && k0 + c < ks;
      copy16(dst + r * kPitch + c, in ? m + (row0 + r) * ld + k0 + c : m, in);
    } else {
      const int r = i / (R / 4), c = i % (R / 4) * 4;
      const bool in = k0 + r < ks && row0 + c < rows;
      copy16(dst + r * (R + 4) + c, in ? m + (k0 + r) * ld + row0 + c : m, in);
    }
  }
}
// Four features (i) x four reduction elements (k) from kk on.
template <int R, bool K_MAJOR>
__device__ __forceinline__ void read_tile(const float *src, int t, int kk, float (&v)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 x = K_MAJOR ? *reinterpret_cast<const float4 *>(src + (t + i * (R / 4)) * kPitch + kk)
                             : *reinterpret_cast<const float4 *>(src + (kk + i) * (R + 4) + t * 4);
    const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) (K_MAJOR ? v[i][j] : v[j][i]) = f[j];
  }
}

// M side: rows of the group (NT, NN) or features of dy (TN); N side: output columns.
template <Mode MODE>
__global__ void __launch_bounds__(kThreads) grouped_f32(int rows, int N, int K, int E,
                                                        const int32_t *__restrict__ offsets,
                                                        const float *__restrict__ A, const float *__restrict__ B,
                                                        const float *__restrict__ row_weight, int accumulate,
                                                        float *out) {
  __shared__ __align__(16) float As[kStages][A_FLOATS];
  __shared__ __align__(16) float Bs[kStages][B_FLOATS];
  __shared__ int start[MODE == TN ? 1 : MAX_E + 1];

  int e, m0, n0 = blockIdx.y * BN, m_end, red, row0;
  if (MODE == TN) {
    e = blockIdx.z;
    row0 = offsets ? offsets[e] : 0;
    const int end = offsets ? offsets[e + 1] : rows;
    if (kChecked && (row0 < 0 || end < row0)) {
      if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) note_violation();
      return;
    }
    row0 = min(max(row0, 0), rows);
    m0 = blockIdx.x * BM;
    m_end = N;
    red = max(min(end, rows) - row0, 0);
    if (red == 0 && accumulate) return;
  } else {
    int *off = reinterpret_cast<int *>(&As[0][0]);  // before the stages need the space
    load_offsets(offsets, rows, E, off);
    __syncthreads();
    if (threadIdx.x < 32) {
      const bool ok = scan_tiles(off, E, rows, BM, start);
      if (kChecked && !ok && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) note_violation();
    }
    __syncthreads();
    if ((int)blockIdx.x >= start[E]) return;
    e = find_group(start, E, 1, blockIdx.x);
    row0 = off[e];
    m0 = row0 + ((int)blockIdx.x - start[e]) * BM;
    m_end = row0 + group_rows(off, e);
    red = K;
    __syncthreads();
  }
  const float *We = MODE == TN ? nullptr : B + (long)e * N * K;
  auto copy = [&](int i) {
    float *a = As[i % kStages], *b = Bs[i % kStages];
    if (MODE == TN) {
      copy_tile<BM, false>(a, A, m0, (long)row0 + i * BK, N, (long)row0 + red, N);
      copy_tile<BN, false>(b, B, n0, (long)row0 + i * BK, K, (long)row0 + red, K);
    } else {
      copy_tile<BM, true>(a, A, m0, i * BK, m_end, K, K);
      if (MODE == NT) copy_tile<BN, true>(b, We, n0, i * BK, N, K, K);
      else copy_tile<BN, false>(b, We, n0, i * BK, N, K, N);
    }
  };

  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  const int steps = (red + BK - 1) / BK;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < steps) copy(i);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  for (int i = 0; i < steps; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncthreads();  // stage i is complete for all, and stage i - 1 read by all
    if (i + kStages - 1 < steps) copy(i + kStages - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    const float *a = As[i % kStages], *b = Bs[i % kStages];
#pragma unroll 2
    for (int kk = 0; kk < BK; kk += 4) {
      float av[4][4], bv[4][4];
      read_tile<BM, MODE != TN>(a, ty, kk, av);
      read_tile<BN, MODE == NT>(b, tx, kk, bv);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) acc[x][y] = fmaf(av[x][k], bv[y][k], acc[x][y]);
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");

  const int ld = MODE == TN ? K : N;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int r = m0 + (MODE != TN ? ty + x * (BM / 4) : ty * 4 + x);
    if (r >= m_end) continue;
    const float w = MODE != TN && row_weight ? row_weight[r] : 1.0f;
    float *dst = out + ((MODE == TN ? (long)e * N : 0l) + r) * ld;
    if (MODE == NT) {
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int col = n0 + tx + y * (BN / 4);
        if (col < ld) dst[col] = acc[x][y] * w;
      }
    } else {
      const int col = n0 + tx * 4;
      if (col >= ld) continue;
      float4 v = make_float4(acc[x][0] * w, acc[x][1] * w, acc[x][2] * w, acc[x][3] * w);
      float4 *o = reinterpret_cast<float4 *>(dst + col);
      if (MODE == TN && accumulate) {
        const float4 old = *o;
        v = make_float4(old.x + v.x, old.y + v.y, old.z + v.z, old.w + v.w);
      }
      *o = v;
    }
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
    grouped_f32<NN><<<grid, kThreads, 0, s>>>(g.rows, g.n, g.k, g.groups, offsets, (const float *)a, (const float *)w,
                                         row_weight, 0, (float *)y);
  else
    grouped_f32<NT><<<grid, kThreads, 0, s>>>(g.rows, g.n, g.k, g.groups, offsets, (const float *)a, (const float *)w,
                                         row_weight, 0, (float *)y);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

moe_status launch_grouped_wgrad_f32(const MoEGrouped &g, const void *dy, const void *a, const int32_t *offsets,
                                    bool accumulate, void *dw, cudaStream_t s) {
  const long nt = (g.k + BN - 1) / BN;
  if (nt > 65535) return MOE_ERR_UNSUPPORTED;
  dim3 grid((unsigned)((g.n + BM - 1) / BM), (unsigned)nt, (unsigned)g.groups);
  grouped_f32<TN><<<grid, kThreads, 0, s>>>(g.rows, g.n, g.k, g.groups, offsets, (const float *)dy, (const float *)a,
                                       nullptr, accumulate, (float *)dw);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
