// What the grouped products (gemm_grouped.cu, gemm_grouped_fp4.cu,
// gemm_grouped_f32.cu) share: bounded waits of the tensor-core pipelines and
// the rows of a group.  Internal to libmoe_b200.
#pragma once

#include <atomic>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace grouped {

constexpr int MAX_E = 1024;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr uint64_t kDrainLimitNs = 200000000ull;  // 0.2 s

// Bounded wait; false if the CTA is aborting (this thread may have started
// it).  The thread sleeps on the barrier with a suspend-time hint: measured
// 2-12% faster over the grouped products than polling it.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, int *abort_flag, int *status) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (;;) {
    if (ptx::mbar_try_wait_sleep(bar, parity, ptx::kWaitHintNs)) return true;
    if (*(volatile int *)abort_flag) return false;
    if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
      *(volatile int *)abort_flag = 1;
      atomicExch(status, kDevTimeout);
      return false;
    }
  }
}

// Warp-uniform wait: every lane waits, and all go on or none.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int *abort_flag, int *status) {
  const bool ok = wait_bar(bar, parity, abort_flag, status);
  return __all_sync(0xffffffffu, ok);
}

// True in one lane of a converged warp, the same one every time.  The
// producer and the MMA issuer run their whole loops under it: known to be one
// thread, the compiler keeps the operands of copies and MMAs in uniform
// registers and issues them without a vote.  With the state of the next stage's
// barrier read ahead of the MMAs (peek), an issue loop of 4 MMAs a stage takes
// 245 cycles, against 395 with a vote, an election and a wait per stage and 650
// under `lane == 0`; 4 MMAs of N = 128 take 256 cycles, of N = 256 512 (one CTA
// an SM, nothing to wait for).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// Used while winding down: copies and MMAs already issued must land first.
__device__ __forceinline__ void drain_bar(uint64_t *bar, uint32_t parity, int *status) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (ptx::globaltimer_ns() - t0 > kDrainLimitNs) {
      atomicExch(status, kDevTimeout);
      return;
    }
  }
}

// Per device and kernel, asked for once (host): the SM count, room for the
// kernel's dynamic shared memory, and the 2-CTA clusters that are resident at
// once (0 for kernels without clusters).  These calls and the tensor maps were
// most of the host time of a small product.
constexpr int kMaxDevices = 64;
struct Launch {
  int sms = 0, pairs = 0;
};
template <typename K>
inline moe_status prepare_launch(K kern, int threads, size_t smem, bool pair, std::atomic<uint64_t> (&known)[kMaxDevices],
                                 Launch &l) {
  int dev = 0;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  const bool cached = dev >= 0 && dev < kMaxDevices;
  uint64_t v = cached ? known[dev].load(std::memory_order_acquire) : 0;
  if (!v) {
    int sms = 0, pairs = 0;
    MOE_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    MOE_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    if (pair) {
      cudaLaunchConfig_t lc = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      lc.gridDim = dim3(2);
      lc.blockDim = dim3(threads);
      lc.dynamicSmemBytes = smem;
      lc.attrs = attr;
      lc.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&pairs, kern, &lc) != cudaSuccess || pairs <= 0) pairs = sms / 2;
    }
    v = ((uint64_t)pairs << 32) | (uint32_t)sms;
    if (cached) known[dev].store(v, std::memory_order_release);
  }
  l.sms = (int)(uint32_t)v;
  l.pairs = (int)(v >> 32);
  return MOE_OK;
}

// Place in a ring of N stages: the stage and the parity of its current round.
template <int N>
struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      ph ^= 1u;
    }
  }
};

// Rows [begin, end) of group e, kept within [0, rows] whatever the offsets
// hold, so that offsets out of range cannot lead to an access out of range.
// offsets == null: one group of all rows.
__device__ __forceinline__ int clamp_row(int v, int rows) { return v < 0 ? 0 : (v > rows ? rows : v); }
__device__ __forceinline__ int seg_begin(const int32_t *offsets, int rows, int e) {
  return offsets ? clamp_row(offsets[e], rows) : 0;
}
__device__ __forceinline__ int seg_end(const int32_t *offsets, int rows, int e) {
  return offsets ? clamp_row(offsets[e + 1], rows) : rows;
}

// One warp: start[e] = sum over e' < e of ceil(rows_e' / tile_rows), e = 0..E
// (the last entry is the total).  Checked build: false if an offset is below
// 0 or the offsets decrease, and then every group counts as empty.
__device__ __forceinline__ bool scan_tiles(const int32_t *offsets, int rows, int E, int tile_rows, int *start) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  bool bad = false;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    int v = 0;
    if (e < E) {
      const int n = seg_end(offsets, rows, e) - seg_begin(offsets, rows, e);
      if (kChecked && offsets && (offsets[e] < 0 || offsets[e + 1] < offsets[e])) bad = true;
      v = n > 0 ? (n + tile_rows - 1) / tile_rows : 0;
    }
    int incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    if (e < E) start[e] = carry + incl - v;
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  const bool any_bad = kChecked && __any_sync(0xffffffffu, bad);
  if (any_bad) {
    for (int e = lane; e < E; e += 32) start[e] = 0;
    carry = 0;
  }
  if (lane == 0) start[E] = carry;
  return !any_bad;
}

// Largest e with start[e] * per <= t (empty groups share the next start).
__device__ __forceinline__ int find_group(const int *start, int E, int per, int t) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] * per <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A tile of tokens: group e's rows are cut into as few tiles of at most
// tile_rows as hold them, of nearly equal widths (multiples of `step`, that of
// the MMA's N), so that 300 rows are 160 + 140 and not 256 + 44: the copies of
// a narrow tile's weights would outlast its MMAs.
struct TokenTile {
  int e, blk, row0, count;  // group, output-feature block, first row, rows
};
__device__ __forceinline__ TokenTile token_tile(const int *start, const int32_t *offsets, int rows, int E, int blocks,
                                                int t, int step) {
  TokenTile r;
  r.e = find_group(start, E, blocks, t);
  const int tiles = start[r.e + 1] - start[r.e];
  const int local = t - start[r.e] * blocks;
  r.blk = local / tiles;
  const int j = local - r.blk * tiles;
  const int begin = seg_begin(offsets, rows, r.e), end = seg_end(offsets, rows, r.e);
  const int width = ((end - begin + tiles - 1) / tiles + step - 1) & ~(step - 1);
  r.row0 = begin + j * width;
  r.count = end - r.row0 < width ? end - r.row0 : width;
  return r;
}

}  // namespace grouped
}  // namespace moe
