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
constexpr uint64_t kStepNs = 4000;                // a stage of a reduction takes 0.2-0.3 us, under 1 when bound by HBM

// Bounded wait; false if the CTA is aborting (this thread may have started
// it).  `steps`: stages of a reduction that pass meanwhile, for the waits that span
// more than one: an epilogue waits for a whole reduction, the clearing warp of a
// weight gradient for the next tile with a partial block.  600 million rows of 8
// columns in one tile take 2.3 s, a healthy launch; so the limit grows by kStepNs a
// stage.  The waits for one stage keep the 2 s.  (A count of issued stages that
// restarts the limit cost 0.5-1% of every product.)  The thread sleeps on the
// barrier with a suspend-time hint: measured 2-12% faster over the grouped products
// than polling it.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, int *abort_flag, int *status,
                                         uint32_t steps = 0) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (;;) {
    if (ptx::mbar_try_wait_sleep(bar, parity, ptx::kWaitHintNs)) return true;
    if (*(volatile int *)abort_flag) return false;
    if (ptx::globaltimer_ns() - t0 > kWaitLimitNs + steps * kStepNs) {
      *(volatile int *)abort_flag = 1;
      atomicExch(status, kDevTimeout);
      return false;
    }
  }
}

// Warp-uniform wait: every lane waits, and all go on or none.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int *abort_flag, int *status,
                                          uint32_t steps = 0) {
  const bool ok = wait_bar(bar, parity, abort_flag, status, steps);
  return __all_sync(0xffffffffu, ok);
}

// True in one lane of a converged warp, the same one every time.  The
// producer and the MMA issuer run their whole loops under it.  With the state of the
// next stage's barrier read ahead of the MMAs, an issue loop of 4 MMAs a stage takes
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

// The epilogue's hand-back of an accumulator to the pair's leader.  It publishes
// no memory: the TMEM reads before it are complete (tcgen05.wait::ld) and ordered
// by tcgen05.fence::before_thread_sync.  A releasing arrive at cluster scope would
// wait for all of the tile's global stores as well, about 2500 cycles a tile
// (weight gradient of 110 rows, 6 x 6128 x 3768: 127 -> 88 us; 23203 rows x 1792
// x 96: 51 -> 45; where the reduction hides it, as in the large products, equal).
__device__ __forceinline__ void arrive_cluster_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
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

// Group offsets to shared memory, off[0..E], by all threads of the block (then a
// barrier): one load latency whatever E, where a warp that scanned them from
// global memory took 10 us for 384 groups.  They are kept within [0, rows], so
// that offsets out of range cannot lead to an access out of range.  offsets ==
// null: one group of all rows.  The checked build keeps negative ones for scan_tiles
// to find.
__device__ __forceinline__ void load_offsets(const int32_t *offsets, int rows, int E, int *off) {
#pragma unroll 4
  for (int e = threadIdx.x; e <= E; e += blockDim.x) {
    const int v = offsets ? offsets[e] : (e ? rows : 0);
    off[e] = kChecked ? (v > rows ? rows : v) : (v < 0 ? 0 : (v > rows ? rows : v));
  }
}
// Rows of group e; 0 if the offsets decrease.
__device__ __forceinline__ int group_rows(const int *off, int e) {
  const int n = off[e + 1] - off[e];
  return n > 0 ? n : 0;
}

// One warp: start[e] = sum over e' < e of ceil(rows_e' / tile_rows), e = 0..E
// (the last entry is the total).  False if the offsets are bad; then all groups are
// empty.  Offsets that decrease make groups overlap, and overlapping groups can have
// more tiles than the host made room for, or than an int counts (1000 groups that
// go to and fro over a million rows): such a call does nothing.  Sums stop just
// above the limit, so that they stay within 32 bits.  Checked build: any negative
// or decreasing offset is bad.
__device__ __forceinline__ bool scan_tiles(int *off, int E, int rows, int tile_rows, int *start) {
  const int lane = threadIdx.x & 31;
  const int limit = (rows + tile_rows - 1) / tile_rows + min(rows, E);
  bool bad = false;
  if (kChecked) {
    for (int e = lane; e < E; e += 32) bad |= off[e] < 0 || off[e + 1] < off[e];
    bad = __any_sync(0xffffffffu, bad);
  }
  // a lane's groups in a row, then one scan over the lanes
  const int per = (E + 31) / 32, e0 = min(lane * per, E), e1 = min(e0 + per, E);
  int sum = 0;
#pragma unroll 4
  for (int e = e0; e < e1; ++e) {
    start[e] = sum;
    sum = min(sum + (group_rows(off, e) + tile_rows - 1) / tile_rows, limit + 1);
  }
  int incl = sum;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, s);
    if (lane >= s) incl += o;
  }
#pragma unroll 4
  for (int e = e0; e < e1; ++e) start[e] += incl - sum;
  if (lane == 31) start[E] = incl;
  bad |= __shfl_sync(0xffffffffu, incl, 31) > limit;
  if (bad) {
    __syncwarp();
    for (int e = lane; e <= E; e += 32) off[e] = start[e] = 0;
  }
  return !bad;
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
__device__ __forceinline__ TokenTile token_tile(const int *start, const int *off, int E, int blocks, int t, int step) {
  TokenTile r;
  r.e = find_group(start, E, blocks, t);
  const int tiles = start[r.e + 1] - start[r.e];
  const int local = t - start[r.e] * blocks;
  r.blk = local / tiles;
  const int j = local - r.blk * tiles;
  const int begin = off[r.e], n = group_rows(off, r.e);
  const int width = ((n + tiles - 1) / tiles + step - 1) & ~(step - 1);
  r.row0 = begin + j * width;
  r.count = n - j * width < width ? n - j * width : width;
  return r;
}

// ---------------------------------------------------------------- epilogue
// Eight warps store a tile of 128 output features (TMEM lanes) x `count` tokens
// (columns) to rows of y [rows, N]: two groups of four, a warp a lane quadrant,
// that take turns at 32 tokens.  (One group took 925 cycles per 32 tokens, the
// dependent latencies of one warp a scheduler; a tile of 256 tokens with a short
// reduction, K = 96, was bound by that.)
//
// bf16: a lane holds one feature of 32 tokens.  It packs two tokens at a time
// and trades with its neighbour, after which the even lane holds features (n,
// n + 1) of the first and the odd lane (n - 1, n) of the second; the four warps
// put 32 tokens x 128 features into shared memory (256 bytes a token; the
// 64-byte quarter of warp q of token t at q ^ (t & 1), so that the two tokens of
// a store take all banks), and each warp writes whole 256-byte rows of 8 tokens.
// fp32: a warp's store is 128 bytes of a row as it is.
constexpr int kRowStage = 2 * 32 * 256;  // bytes: a buffer a group
constexpr int kEpiGroups = 2;
// Named barriers of the epilogue: 1 and 2 for the groups, 3 for all its warps; 4
// and 5 for the scale warps of gemm_grouped_fp4.cu.
__device__ __forceinline__ void epi_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }
// The same decision for all `threads` of the barrier: true if `ok` is in every one.
template <int BARRIER, int THREADS>
__device__ __forceinline__ bool all_agree(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)ok), "n"(BARRIER), "n"(THREADS)
      : "memory");
  return r != 0;
}

struct RowStore {
  void *out;
  int out_f32;
  int N;
  const float *w0, *w1;  // factors of a row [rows], or null
};

// ---------------------------------------------------------------- split sums
// A tile whose reduction is cut into parts: every part's CTA leaves its sums in
// its shared memory and the CTAs of the cluster add them, in the parts' order,
// four neighbours of the output a thread, several quads' loads in flight (one
// load after the other took 10 us for 64 x 128 sums of two parts, this 1-2).
//   by column  [column][feature], pitch 132: tokens x features
//   by feature [feature][column], pitch columns + 4: rows of dW
constexpr int kColPitch = 132;

// Warps of group `group` of `groups` take every groups-th run of 32 columns.
__device__ __forceinline__ void put_part_columns(float *parts, uint32_t tbase, int count, int q, int group, int groups) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int c = group * 32; c < count; c += groups * 32) {
    uint32_t v[32];
    ptx::tmem_ld32(tbase + c, v);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (c + j < count) parts[(c + j) * kColPitch + q * 32 + lane] = __uint_as_float(v[j]);
  }
}
__device__ __forceinline__ void put_part_features(float *parts, uint32_t tbase, int count, int pitch, int q) {
  float *row = parts + (q * 32 + (threadIdx.x & 31)) * pitch;
#pragma unroll 1
  for (int c = 0; c < count; c += 32) {
    uint32_t v[32];
    ptx::tmem_ld32(tbase + c, v);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; j += 4)
      if (c + j < count) *reinterpret_cast<uint4 *>(row + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
  }
}

// Sums of the quads at parts + at[u] over the CTAs first, first + step, ... of
// the cluster (`n` of them, only those with `has` bit set), U quads at once.
template <int U>
__device__ __forceinline__ void add_parts(const float *parts, const int (&at)[U], uint32_t first, uint32_t step, int n,
                                          uint32_t has, float4 (&sum)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) sum[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int k = 0; k < n; ++k) {
    if (!(has >> k & 1)) continue;
    const uint32_t base = ptx::map_to_rank(parts, first + k * step);
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[u].x), "=f"(v[u].y), "=f"(v[u].z), "=f"(v[u].w)
                   : "r"(base + (uint32_t)at[u] * 4u));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      sum[u].x += v[u].x;
      sum[u].y += v[u].y;
      sum[u].z += v[u].z;
      sum[u].w += v[u].w;
    }
  }
}
__device__ __forceinline__ void put_quad(void *out, int out_f32, long at, float4 v, bool accumulate) {
  if (out_f32) {
    float4 *o = reinterpret_cast<float4 *>((float *)out + at);
    if (accumulate) {
      const float4 old = *o;
      v = make_float4(old.x + v.x, old.y + v.y, old.z + v.z, old.w + v.w);
    }
    *o = v;
  } else {  // rounded once
    uint2 *o = reinterpret_cast<uint2 *>((__nv_bfloat16 *)out + at);
    if (accumulate) {
      const uint2 old = *o;
      const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&old.x));
      const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&old.y));
      v = make_float4(a.x + v.x, a.y + v.y, b.x + v.z, b.y + v.w);
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *o = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
  }
}
// This CTA's share of a tile of tokens: tokens [c_lo, c_lo + w) x 128 features from n0 on.
__device__ __forceinline__ void store_summed_tokens(const RowStore &o, const float *parts, int row0, int c_lo, int w,
                                                    int n0, const float *feature_scale, uint32_t first, uint32_t step,
                                                    int n, uint32_t has, int threads) {
  constexpr int U = 4;
  const int quads = w * 32;
  for (int i0 = threadIdx.x; i0 < quads; i0 += U * threads) {
    int at[U];
    float4 sum[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u * threads, quads - 1);
      at[u] = (c_lo + (i >> 5)) * kColPitch + (i & 31) * 4;
    }
    add_parts(parts, at, first, step, n, has, sum);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * threads, r = row0 + c_lo + (i >> 5), f = n0 + (i & 31) * 4;
      if (i >= quads || f >= o.N) continue;
      float4 v = sum[u];
      if (feature_scale) {
        const float *s = feature_scale + f;
        v = make_float4(v.x * s[0], v.y * s[1], v.z * s[2], v.w * s[3]);
      }
      float k = 1.0f;
      if (o.w0) k = o.w0[r];
      if (o.w1) k *= o.w1[r];
      put_quad(o.out, o.out_f32, (long)r * o.N + f, make_float4(v.x * k, v.y * k, v.z * k, v.w * k), false);
    }
  }
}

// The factor of a tile's token c + lane.  Read a round ahead of its use (the
// first before the wait for the tile), so that its latency is not paid a round
// after the other (23203 rows x 1792 x 96 over 20 groups: 74 -> 61 us).
__device__ __forceinline__ float row_factor(const RowStore &o, int row0, int count, int c) {
  const int t = c + (threadIdx.x & 31);
  float w = 1.0f;
  if (t < count) {
    if (o.w0) w = o.w0[row0 + t];
    if (o.w1) w *= o.w1[row0 + t];
  }
  return w;
}

// q: this warp's lane quadrant; n0: the tile's first feature; w: row_factor of
// the group's first round; SCALED: times `scale`, this lane's feature factor.
// stage: kRowStage bytes; wbuf: 32 floats of this warp's.
template <bool SCALED>
__device__ __forceinline__ void store_tokens(const RowStore &o, uint32_t tbase, int row0, int count, int n0, int q,
                                             int group, float w, float scale, uint8_t *stage, float *wbuf) {
  const int lane = threadIdx.x & 31;
  const int n = n0 + q * 32 + lane;
  const bool weighted = o.w0 || o.w1;
  const int odd = lane & 1;
  constexpr int step = 32 * kEpiGroups;
  if (group * 32 >= count) return;  // all four warps of the group
  uint8_t *buf = stage + group * (kRowStage / kEpiGroups);
  uint32_t v[32];
  ptx::tmem_ld32(tbase + group * 32, v);
#pragma unroll 1
  for (int c = group * 32; c < count; c += step) {
    const int left = count - c;
    if (weighted) {
      __syncwarp();
      wbuf[lane] = w;
      __syncwarp();
      if (c + step < count) w = row_factor(o, row0, count, c + step);
    }
    ptx::tmem_ld_wait();
    float f[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) f[j] = SCALED ? __uint_as_float(v[j]) * scale : __uint_as_float(v[j]);
    if (weighted) {
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 k = *reinterpret_cast<const float4 *>(wbuf + j);
        f[j] *= k.x, f[j + 1] *= k.y, f[j + 2] *= k.z, f[j + 3] *= k.w;
      }
    }
    if (c + step < count) ptx::tmem_ld32(tbase + c + step, v);
    if (o.out_f32) {
      float *y = (float *)o.out + (long)(row0 + c) * o.N + n;
      if (n < o.N) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < left) y[(long)j * o.N] = f[j];
      }
      continue;
    }
    if (c != group * 32) epi_sync(group);  // the round before has been read
    uint8_t *at = buf + odd * 256 + ((q ^ odd) << 6) + ((lane & ~1) << 1);
    const uint32_t pick = odd ? 0x3276u : 0x5410u;  // odd: (other's high, own high), even: (own low, other's low)
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(f[j], f[j + 1]);
      const uint32_t own = *reinterpret_cast<const uint32_t *>(&p);
      const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
      *reinterpret_cast<uint32_t *>(at + j * 256) = __byte_perm(own, other, pick);
    }
    epi_sync(group);
    // this warp's 8 tokens, two a round: 16 lanes x 16 bytes each
    const int piece = lane & 15, half = lane >> 4;
    const bool in = n0 + piece * 8 < o.N;
    uint4 rows[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = q * 8 + 2 * i + half;
      rows[i] = *reinterpret_cast<const uint4 *>(buf + t * 256 + (((piece >> 2) ^ (t & 1)) << 6) + ((piece & 3) << 4));
    }
    __nv_bfloat16 *y = (__nv_bfloat16 *)o.out + (long)(row0 + c + q * 8 + half) * o.N + n0 + piece * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (in && q * 8 + 2 * i + half < left) *reinterpret_cast<uint4 *>(y + (long)(2 * i) * o.N) = rows[i];
  }
  if (!o.out_f32) epi_sync(group);  // read before the next tile's first round
}

}  // namespace grouped
}  // namespace moe
