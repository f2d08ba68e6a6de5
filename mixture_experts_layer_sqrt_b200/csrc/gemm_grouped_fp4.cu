// Product of two NVFP4 operands grouped by expert (tcgen05 block-scaled MMA):
//
//   y[r, n] = w_r * ra_r * rw_en * sum_k (qa[r, k] sa[r, k/16]) (qw[e, n, k] sw[e, n, k/16])
//
// for the rows r of group e: e2m1 codes q, an e4m3 scale per 16 of them, and
// optional fp32 row scales of either operand.  The MMA multiplies codes and
// scales exactly and accumulates in fp32; the row scales and the routing
// weight enter in the epilogue.
//
// Layout of the work as in gemm_grouped.cu: weights on the MMA's M side (128
// output features a tile), the tokens of one group on its N side (up to BT,
// rounded to 16), so ragged groups pad few columns and no rows, and the packed
// weights are read once per BT tokens.  A stage of codes holds 256 reduction elements, rows of
// 128 bytes (128-byte swizzle); a stage of scales those of four of them, rows of
// 64 bytes (64-byte swizzle).  TMA's cost is by the row here: 49152 rows x 4096
// x 2048 over 384 groups took 418-427 us with 16 bytes of scales a row and
// stage, 417 with 32, 399 with 64.
//
// A scale's sign bit is not read by the MMA (0xB8 counts as 1).  Looking for one in
// the scale warps took 1-5% (NVFP4 prefill 396 -> 408 us, 8192 x 4096 x 2048 over 64
// groups 75.5 -> 77.5), replacing what they found 4-37%: the header defines it away.
//
// The MMA takes the scales from TMEM: for each 64 reduction elements one
// 32-bit column per 32 rows (lane i of column j: the four scale bytes of row
// 32 j + i), the same in all four lane quadrants.  Four warps, one a quadrant,
// copy them there from the stage with tcgen05.st, one 16-byte read a row, up to
// SF_BUFS stages ahead of the MMAs.  Scale rows that TMA cannot read (K not a
// multiple of 256: rows not a multiple of 16 bytes) are copied by the same warps.
//
// Roles (480 threads, persistent, one CTA per SM): warp 0 TMA producer of the
// weights, warp 1 TMEM owner and MMA issuer, warps 2-9 epilogue, warps 10-13
// scales, warp 14 TMA producer of the tokens.  Every wait is bounded.
//
// Measured (B200): 48 rows x 4096 x 2048 over 384 groups 46 us (227 MB of weights
// at 4.9 TB/s; the last tiles, with five or six a CTA, and the start take the
// rest); 49152 rows 383-407 us (2.1 GB, 5.4 TB/s), 464 us after a second under the
// power limit; 8192 rows x 4096 x 4096 over 4 groups 89 us = 3.1 PFLOP/s.
#include <cudaTypedefs.h>
#include <limits.h>

#include "grouped.cuh"
#include "kernels.h"
#include "tma_host.h"

namespace moe {

MOE_VIOLATION_COUNTER(violations_gemm_grouped_fp4)

namespace {

using namespace grouped;

constexpr int BM = 128;                 // output features per tile
constexpr int BK = 256;                 // reduction elements per stage
constexpr int ROW = BK / 2;             // bytes of codes a row and stage
constexpr int MMA_K = 64;
constexpr int STEPS = BK / MMA_K;
constexpr int TOK_BOX = 32;             // token rows per TMA box
constexpr int SPAN = 4;                 // stages of codes that a stage of scales covers
constexpr int SROW = 16 * SPAN;         // its bytes a row
constexpr int S_STAGES = 2;
constexpr int kRawSpan = 2;             // and of raw scale rows, the path without TMA
constexpr int kRawRow = 16 * (kRawSpan + 1);
constexpr int kThreads = 480;
constexpr int kScaleWarp0 = 10;
constexpr int kTokenWarp = 14;

template <int BT, bool SF_TMA>
struct Cfg {
  static constexpr int A_BYTES = BM * ROW, B_BYTES = BT * ROW;  // codes of a stage
  // Rings of their own: the weights come from DRAM, the tokens mostly from L2.
  static constexpr int A_STAGES = (BT == 192 ? 4 : 8) - (SF_TMA ? 0 : 1);
  static constexpr int B_STAGES = BT == 192 ? 4 : 5;
  static constexpr int S_BYTES = (BM + BT) * SROW;              // scales of SPAN stages
  // without TMA: stages of raw scale rows, in the space of these and of a weight stage
  static constexpr int RAW_STAGES = 3;
  static constexpr int RAW_BYTES = (BM + BT) * kRawRow;
  static constexpr int ROWS_BYTES = (BM + BT) * 16 * kRawSpan;  // one of them in place
  static constexpr int BYTES =
      A_STAGES * A_BYTES + B_STAGES * B_BYTES + (SF_TMA ? S_STAGES * S_BYTES : RAW_STAGES * RAW_BYTES + ROWS_BYTES);
  static constexpr int SFA_COLS = STEPS * BM / 32;   // TMEM columns of a stage's scales
  static constexpr int SFB_COLS = STEPS * BT / 32;
  static constexpr int SF_COLS = SFA_COLS + SFB_COLS;
  static constexpr int SF_BUFS = BT == 192 ? 3 : 4;  // stages' scales in TMEM at once
  static constexpr int SF_BASE = 2 * BT;             // past the two accumulators
  static constexpr uint32_t TMEM_COLS = BT == 192 ? 512 : 256;
  static_assert(SF_BASE + SF_BUFS * SF_COLS <= (int)TMEM_COLS, "accumulators and scales fit in TMEM");
};

struct Smem {
  uint64_t a_full[8], a_empty[8];                    // weight codes
  uint64_t b_full[8], b_empty[8];                    // token codes
  uint64_t s_full[S_STAGES], s_empty[S_STAGES];      // scales of both
  uint64_t sf_full[4];
  uint64_t sf_empty[4];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint64_t drain;
  __align__(16) float wbuf[4 * kEpiGroups * 32];  // row factors, 32 an epilogue warp
  uint32_t tmem_base;
  int abort;
  int start[MAX_E + 1];
  int off[MAX_E + 1];
};
constexpr int kSmemPart = 9728;
static_assert(sizeof(Smem) <= kSmemPart, "barriers and tile list");

struct Params {
  int rows, N, K, E, m_blocks;
  int tile;   // tokens of a tile, at most BT
  int split;  // parts that a tile's reduction is cut into, one a CTA of a cluster
  const int32_t *offsets;
  const uint8_t *sa, *sw;     // scale rows, for the path without TMA
  const float *ra, *rw;       // row scales [rows], [E, N], or null
  const float *row_weight;    // [rows] or null
  void *out;
  int out_f32;
  int *status;
};

// D (+)= (A sfA) (B sfB)^T: e2m1 operands, an e4m3 scale per 16; one thread issues.
__device__ __forceinline__ void mma_nvfp4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// This thread's TMEM lane, consecutive columns.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Instruction descriptor of kind::mxf4nvf4 without N: A and B e2m1 (code 1 at
// [7,10) and [10,12)), both K-major, e4m3 scales (bit 23 = 0), M >> 7 at
// [27,29), scale data ids 0, K = 64 (bit 31 = 0).
constexpr uint32_t kIdesc0 = (1u << 7) | (1u << 10) | ((uint32_t)(BM >> 7) << 27);

// Scale rows that TMA cannot read start at any even byte.  The scale warps copy
// the aligned 16-byte chunks that hold a row's next kRawSpan stages (three) as
// they are, asynchronously, two such runs ahead, and then shift them into place, a
// row a thread.  (Loads into registers instead of the copies took 155 us for 8262
// rows x 2080 x 2040 over 67 groups, a shift by every warp that reads them 128.)
// 16 bytes to shared memory, the first `bytes` of them read and the others zero.
__device__ __forceinline__ void copy_chunk(void *dst, const uint8_t *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_addr(dst)), "l"(src), "r"(bytes)
               : "memory");
}
// 16 bytes from byte `shift` (even, < 16) of two chunks on, those from `left` on zero.
__device__ __forceinline__ void shifted(const uint8_t *chunks, int shift, int left, uint32_t (&v)[4]) {
  const uint4 lo = reinterpret_cast<const uint4 *>(chunks)[0], hi = reinterpret_cast<const uint4 *>(chunks)[1];
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t u[6], t[5];
#pragma unroll
  for (int i = 0; i < 6; ++i) u[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) t[i] = shift & 4 ? u[i + 1] : u[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(t[i], t[i + 1], (shift & 2) * 8);
  if (left < 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * i + 2 >= left) v[i] &= 0xFFFFu;
      if (4 * i >= left) v[i] = 0;
    }
  }
}

template <int BT, bool SF_TMA>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_fp4(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                     const Params p) {
  using C = Cfg<BT, SF_TMA>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *stage_a = base;
  uint8_t *stage_b = stage_a + C::A_STAGES * C::A_BYTES;
  uint8_t *stage_s = stage_b + C::B_STAGES * C::B_BYTES;  // rows of the weights, then of the tokens
  Smem &sm = *reinterpret_cast<Smem *>(base + C::BYTES);
  float *parts = reinterpret_cast<float *>(base);  // split: over the stages once the MMAs have read them
  uint8_t *staging = reinterpret_cast<uint8_t *>(&sm) + kSmemPart;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::A_STAGES; ++s) {
      ptx::mbar_init(&sm.a_full[s], 1);
      ptx::mbar_init(&sm.a_empty[s], 1);
    }
    for (int s = 0; s < C::B_STAGES; ++s) {
      ptx::mbar_init(&sm.b_full[s], 1);
      ptx::mbar_init(&sm.b_empty[s], 1);
    }
    for (int s = 0; s < S_STAGES; ++s) {
      ptx::mbar_init(&sm.s_full[s], 2);   // both producers
      ptx::mbar_init(&sm.s_empty[s], 4);  // scale warps
    }
    for (int a = 0; a < C::SF_BUFS; ++a) {
      ptx::mbar_init(&sm.sf_full[a], 4);
      ptx::mbar_init(&sm.sf_empty[a], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&sm.tmem_full[a], 1);
      ptx::mbar_init(&sm.tmem_empty[a], 4 * kEpiGroups);
    }
    ptx::mbar_init(&sm.drain, 1);
    sm.abort = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
    if (SF_TMA) {
      ptx::prefetch_tmap(&tmSA);
      ptx::prefetch_tmap(&tmSB);
    }
  }
  if (warp == 1) {
    ptx::tmem_alloc(&sm.tmem_base, C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  load_offsets(p.offsets, p.rows, p.E, sm.off);
  __syncthreads();
  if (warp == 2) {
    const bool ok = scan_tiles(sm.off, p.E, p.rows, p.tile, sm.start);
    if (kChecked && !ok && lane == 0 && blockIdx.x == 0) note_violation();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = sm.tmem_base;
  const int total = sm.start[p.E] * p.m_blocks;
  // a cluster's CTAs share a tile, each with its blocks [kb0, kb1) of the reduction
  const int part = (int)ptx::cluster_ctarank();
  const int unit = (int)blockIdx.x / p.split, n_units = (int)gridDim.x / p.split;
  const int blocks = (p.K + BK - 1) / BK;
  const int kb0 = (int)((long)blocks * part / p.split), kb1 = (int)((long)blocks * (part + 1) / p.split);
  auto tile_of = [&](int t) { return token_tile(sm.start, sm.off, p.E, p.m_blocks, t, 16); };

  if (warp == 0 || warp == kTokenWarp) {
    // ================================================= TMA producers: weights, tokens
    const bool weights = warp == 0;
    if (elect_one()) {
      uint64_t *const full = weights ? sm.a_full : sm.b_full, *const empty = weights ? sm.a_empty : sm.b_empty;
      const int stages = weights ? C::A_STAGES : C::B_STAGES;
      int s = 0;
      uint32_t ph = 0, issued = 0, s_issued = 0;
      Ring<S_STAGES> sc;
      bool ok = true;
      for (int t = unit; t < total && ok; t += n_units) {
        const TokenTile tl = tile_of(t);
        const int boxes = (tl.count + TOK_BOX - 1) / TOK_BOX;
        const uint32_t tx = weights ? C::A_BYTES : boxes * TOK_BOX * ROW;
        const uint32_t s_tx = weights ? BM * SROW : boxes * TOK_BOX * SROW;
        for (int kb = kb0; kb < kb1; ++kb, ++issued) {
          if (SF_TMA && (kb - kb0) % SPAN == 0) {
            if (!wait_bar(&sm.s_empty[sc.s], sc.ph ^ 1u, &sm.abort, p.status)) {
              ok = false;
              break;
            }
            uint8_t *d = stage_s + sc.s * C::S_BYTES;
            ptx::mbar_arrive_expect_tx(&sm.s_full[sc.s], s_tx);
            if (weights) {
              ptx::tma_load_3d(d, &tmSA, &sm.s_full[sc.s], kb * 16, tl.blk * BM, tl.e);
            } else {
              for (int i = 0; i < boxes; ++i)
                ptx::tma_load_3d(d + (BM + i * TOK_BOX) * SROW, &tmSB, &sm.s_full[sc.s], kb * 16, tl.row0 + i * TOK_BOX, 0);
            }
            sc.next();
            ++s_issued;
          }
          if (!wait_bar(&empty[s], ph ^ 1u, &sm.abort, p.status)) {
            ok = false;
            break;
          }
          uint64_t *bar = &full[s];
          ptx::mbar_arrive_expect_tx(bar, tx);
          if (weights) {
            ptx::tma_load_3d(stage_a + s * C::A_BYTES, &tmA, bar, kb * ROW, tl.blk * BM, tl.e);
          } else {
            for (int i = 0; i < boxes; ++i)
              ptx::tma_load_3d(stage_b + s * C::B_BYTES + i * TOK_BOX * ROW, &tmB, bar, kb * ROW, tl.row0 + i * TOK_BOX,
                               0);
          }
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // every issued copy has landed before shared memory is released
      for (int i = 0; i < stages && (uint32_t)i < issued; ++i)
        drain_bar(&full[i], (issued - 1 - i) / stages & 1u, p.status);
      for (int i = 0; i < S_STAGES && (uint32_t)i < s_issued; ++i)
        drain_bar(&sm.s_full[i], (s_issued - 1 - i) / S_STAGES & 1u, p.status);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================================================= MMA issuer
    if (elect_one()) {
      const uint64_t ad0 = ptx::desc_kmajor_sw128(ptx::smem_addr(stage_a));
      const uint64_t bd0 = ptx::desc_kmajor_sw128(ptx::smem_addr(stage_b));
      Ring<C::A_STAGES> ra;
      Ring<C::B_STAGES> rb;
      Ring<C::SF_BUFS> sf;
      bool a_ready = false, b_ready = false, sf_ready = false;  // the next stage's barriers, read ahead
      int i = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += n_units, ++i) {
        const TokenTile tl = tile_of(t);
        const int acc = i & 1;
        const uint32_t aph = (i >> 1) & 1u;
        if (!wait_bar(&sm.tmem_empty[acc], aph ^ 1u, &sm.abort, p.status)) break;
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BT;
        const uint32_t idesc = kIdesc0 | (uint32_t)((tl.count + 15) >> 4) << 18;  // N >> 3 at bit 17
        for (int kb = kb0; kb < kb1; ++kb) {
          if ((!a_ready && !wait_bar(&sm.a_full[ra.s], ra.ph, &sm.abort, p.status)) ||
              (!b_ready && !wait_bar(&sm.b_full[rb.s], rb.ph, &sm.abort, p.status)) ||
              (!sf_ready && !wait_bar(&sm.sf_full[sf.s], sf.ph, &sm.abort, p.status))) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const int as = ra.s, bs = rb.s;
          ra.next();
          rb.next();
          Ring<C::SF_BUFS> sn = sf;
          sn.next();
          a_ready = ptx::mbar_try_wait(&sm.a_full[ra.s], ra.ph);
          b_ready = ptx::mbar_try_wait(&sm.b_full[rb.s], rb.ph);
          sf_ready = ptx::mbar_try_wait(&sm.sf_full[sn.s], sn.ph);
          const uint64_t ad = ad0 + (uint32_t)as * (C::A_BYTES >> 4), bd = bd0 + (uint32_t)bs * (C::B_BYTES >> 4);
          const uint32_t sfa = tmem_base + C::SF_BASE + sf.s * C::SF_COLS, sfb = sfa + C::SFA_COLS;
#pragma unroll
          for (int k = 0; k < STEPS; ++k)
            mma_nvfp4(d_tmem, ad + k * (MMA_K / 2 >> 4), bd + k * (MMA_K / 2 >> 4), idesc, sfa + k * (BM / 32),
                      sfb + k * (BT / 32), ((kb - kb0) | k) != 0);
          ptx::mma_commit(&sm.a_empty[as]);
          ptx::mma_commit(&sm.b_empty[bs]);
          ptx::mma_commit(&sm.sf_empty[sf.s]);
          sf = sn;
        }
        if (ok) ptx::mma_commit(&sm.tmem_full[acc]);
      }
      ptx::mma_commit(&sm.drain);
      drain_bar(&sm.drain, 0, p.status);
    }
    __syncwarp();
  } else if (warp >= kScaleWarp0 && warp < kTokenWarp) {
    // ================================================= scales to TMEM
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    constexpr int AR = BM / 32, BR = BT / 32;  // rows of each operand a lane
    Ring<S_STAGES> sc;
    Ring<C::SF_BUFS> sf;
    bool ok = true;
    // the path without TMA
    const int pitch = p.K / 16, tid = threadIdx.x - kScaleWarp0 * 32;
    int raw = 0;  // stage of raw rows to read
    uint8_t *const in_place = stage_s + C::RAW_STAGES * C::RAW_BYTES;
    // the copies run RAW_STAGES - 1 stages ahead, over the tiles' ends
    int c_t = unit, c_kb = kb0, c_stage = 0;
    TokenTile c_tl = {};
    if (!SF_TMA && unit < total) c_tl = tile_of(unit);
    auto copy = [&]() {
      if (c_t < total) {
        // offsets from the tile's first rows, rounded down to a chunk
        const long wt = ((long)c_tl.e * p.N + c_tl.blk * BM) * pitch + c_kb * 16, tk = (long)c_tl.row0 * pitch + c_kb * 16;
        const int left = min(pitch - c_kb * 16, 16 * kRawSpan);
        const uint8_t *const w_at = p.sw + (wt & ~15l), *const t_at = p.sa + (tk & ~15l);
        const int w_mis = (int)(wt & 15), t_mis = (int)(tk & 15);
        const int w_all = (int)min((long)p.E * p.N * pitch - (wt & ~15l), 0x40000000l);
        const int t_all = (int)min((long)p.rows * pitch - (tk & ~15l), 0x40000000l);
        const int w_rows = min(p.N - c_tl.blk * BM, BM), t_rows = c_tl.count;
        uint8_t *const dst = stage_s + c_stage * C::RAW_BYTES;
#pragma unroll 4
        for (int i = tid; i < (BM + BT) * (kRawSpan + 1); i += 128) {
          const int row = i / (kRawSpan + 1), c = i - row * (kRawSpan + 1);
          const bool weight = row < BM;
          const int r = weight ? row : row - BM;
          const int off = r * pitch + (weight ? w_mis : t_mis);
          const int at = (off & ~15) + 16 * c;
          const bool in = r < (weight ? w_rows : t_rows) && 16 * c < (off & 15) + left;
          copy_chunk(dst + i * 16, (weight ? w_at : t_at) + (in ? at : 0), in ? min(16, (weight ? w_all : t_all) - at) : 0);
        }
        c_kb += kRawSpan;
        if (c_kb >= kb1) {
          c_kb = kb0;
          c_t += n_units;
          if (c_t < total) c_tl = tile_of(c_t);
        }
        c_stage = c_stage + 1 == C::RAW_STAGES ? 0 : c_stage + 1;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (!SF_TMA)
      for (int i = 0; i < C::RAW_STAGES - 1; ++i) copy();
    bool leave = false;
    for (int t = unit; t < total && !leave; t += n_units) {
      const TokenTile tl = tile_of(t);
      uint32_t va[AR][4], vb[BR][4];
      const int a_mis = (int)(((long)tl.e * p.N + tl.blk * BM) * pitch & 15);  // of the tile's first rows
      const int b_mis = (int)((long)tl.row0 * pitch & 15);
      for (int kb = kb0; kb < kb1; ++kb, sf.next()) {
        if (SF_TMA) {
          const int at_k = (kb - kb0) % SPAN;  // 16-byte piece of the scale rows
          if (at_k == 0 && !warp_wait(&sm.s_full[sc.s], sc.ph, &sm.abort, p.status)) {
            ok = false;
            leave = true;
            break;
          }
          __syncwarp();
          // rows 64 bytes apart: 16-byte piece c of row r at c ^ (r / 2 % 4) (64-byte swizzle)
          const uint4 *a = reinterpret_cast<const uint4 *>(stage_s + sc.s * C::S_BYTES) + lane * SPAN +
                           (at_k ^ ((lane >> 1) & 3));
          const uint4 *b = a + BM * SPAN;
#pragma unroll
          for (int j = 0; j < AR; ++j) {
            const uint4 v = a[j * 32 * SPAN];
            va[j][0] = v.x, va[j][1] = v.y, va[j][2] = v.z, va[j][3] = v.w;
          }
#pragma unroll
          for (int j = 0; j < BR; ++j) {
            const uint4 v = b[j * 32 * SPAN];
            vb[j][0] = v.x, vb[j][1] = v.y, vb[j][2] = v.z, vb[j][3] = v.w;
          }
          if (at_k == SPAN - 1 || kb == kb1 - 1) {  // the stage's last rows are in registers
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sm.s_empty[sc.s]);
            sc.next();
          }
        } else {
          const int at_k = (kb - kb0) % kRawSpan;
          if (at_k == 0) {
            // the stage has landed for all, and the one before is read by all
            asm volatile("cp.async.wait_group %0;" ::"n"(C::RAW_STAGES - 2) : "memory");
            ok = all_agree<4, 128>(ok);
            if (!ok) {
              leave = true;
              break;
            }
            copy();
            // into place, a row a thread: 16-byte piece c of row r at c ^ (r / 4 % 2)
            const uint8_t *from = stage_s + raw * C::RAW_BYTES;
            raw = raw + 1 == C::RAW_STAGES ? 0 : raw + 1;
            const int left = pitch - kb * 16;
            for (int r = tid; r < BM + BT; r += 128) {
              const int shift = (r < BM ? a_mis + r * pitch : b_mis + (r - BM) * pitch) & 15;
#pragma unroll
              for (int c = 0; c < kRawSpan; ++c) {
                uint32_t v[4];
                shifted(from + r * kRawRow + c * 16, shift, left - c * 16, v);
                *reinterpret_cast<uint4 *>(in_place + r * 16 * kRawSpan + ((c ^ ((r >> 2) & 1)) << 4)) =
                    make_uint4(v[0], v[1], v[2], v[3]);
              }
            }
            asm volatile("bar.sync 5, 128;" ::: "memory");
          }
          const uint4 *a = reinterpret_cast<const uint4 *>(in_place) + lane * kRawSpan + (at_k ^ ((lane >> 2) & 1));
          const uint4 *b = a + BM * kRawSpan;
#pragma unroll
          for (int j = 0; j < AR; ++j) {
            const uint4 v = a[j * 32 * kRawSpan];
            va[j][0] = v.x, va[j][1] = v.y, va[j][2] = v.z, va[j][3] = v.w;
          }
#pragma unroll
          for (int j = 0; j < BR; ++j) {
            const uint4 v = b[j * 32 * kRawSpan];
            vb[j][0] = v.x, vb[j][1] = v.y, vb[j][2] = v.z, vb[j][3] = v.w;
          }
        }
        ok = ok && warp_wait(&sm.sf_empty[sf.s], sf.ph ^ 1u, &sm.abort, p.status);
        if (!ok) {
          leave = SF_TMA;
          if (SF_TMA) break;
          continue;  // without TMA the warps leave together, at the next raw stage
        }
        ptx::tc_fence_after();
        uint32_t ca[C::SFA_COLS], cb[C::SFB_COLS];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
#pragma unroll
          for (int j = 0; j < AR; ++j) ca[k * AR + j] = va[j][k];
#pragma unroll
          for (int j = 0; j < BR; ++j) cb[k * BR + j] = vb[j][k];
        }
        const uint32_t at = tmem_base + lane_addr + C::SF_BASE + sf.s * C::SF_COLS;
#pragma unroll
        for (int c = 0; c < C::SFA_COLS; c += 8) tmem_st8(at + c, ca + c);
#pragma unroll
        for (int c = 0; c < C::SFB_COLS; c += 8) tmem_st8(at + C::SFA_COLS + c, cb + c);
        tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.sf_full[sf.s]);
      }
    }
  } else {
    // ================================================= epilogue (warps 2..9)
    const int q = warp & 3, group = (warp - 2) >> 2;
    const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
    const RowStore store = {p.out, p.out_f32, p.N, p.ra, p.row_weight};
    int i = 0;
    for (int t = unit; t < total; t += n_units, ++i) {
      const TokenTile tl = tile_of(t);
      const int acc = i & 1;
      const uint32_t aph = (i >> 1) & 1u;
      const int n = tl.blk * BM + q * 32 + lane;
      const float w0 = row_factor(store, tl.row0, tl.count, group * 32);
      const float wn = p.rw && n < p.N ? p.rw[(long)tl.e * p.N + n] : 1.0f;
      if (!all_agree<3, 128 * kEpiGroups>(warp_wait(&sm.tmem_full[acc], aph, &sm.abort, p.status, kb1 - kb0))) break;
      ptx::tc_fence_after();
      const uint32_t tbase = tmem_base + lane_addr + acc * BT;
      if (p.split > 1) put_part_columns(parts, tbase, tl.count, q, group, kEpiGroups);
      else store_tokens<true>(store, tbase, tl.row0, tl.count, tl.blk * BM, q, group, w0, wn, staging,
                              sm.wbuf + (warp - 2) * 32);
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.tmem_empty[acc]);
    }
  }

  if (p.split > 1) {
    // the parts' sums, in the parts' order, each part a share of the tokens
    __syncwarp();
    ptx::cluster_sync();
    if (unit < total) {
      const TokenTile tl = tile_of(unit);
      const int c_lo = tl.count * part / p.split, w = tl.count * (part + 1) / p.split - c_lo;
      const RowStore store = {p.out, p.out_f32, p.N, p.ra, p.row_weight};
      store_summed_tokens(store, parts, tl.row0, c_lo, w, tl.blk * BM, p.rw ? p.rw + (long)tl.e * p.N : nullptr, 0, 1,
                          p.split, (1u << p.split) - 1, kThreads);
    }
  }
  ptx::tc_fence_before();
  __syncwarp();
  if (p.split > 1) ptx::cluster_sync();  // no CTA leaves while another reads its sums
  else __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <int BT, bool SF_TMA>
moe_status launch(Params &p, const void *a, const void *w, cudaStream_t s) {
  using C = Cfg<BT, SF_TMA>;
  CUtensorMap ta, tb, tsa, tsb;
  if (!tma_map_u8(&ta, w, (uint64_t)p.K / 2, p.N, p.E, ROW, BM, 128) ||
      !tma_map_u8(&tb, a, (uint64_t)p.K / 2, p.rows, 1, ROW, TOK_BOX, 128))
    return MOE_ERR_CUDA;
  tsa = ta;
  tsb = tb;
  if (SF_TMA && (!tma_map_u8(&tsa, p.sw, (uint64_t)p.K / 16, p.N, p.E, SROW, BM, SROW) ||
                 !tma_map_u8(&tsb, p.sa, (uint64_t)p.K / 16, p.rows, 1, SROW, TOK_BOX, SROW)))
    return MOE_ERR_CUDA;
  const size_t smem = 1024 + (size_t)C::BYTES + kSmemPart + kRowStage;
  auto kern = grouped_gemm_fp4<BT, SF_TMA>;
  static std::atomic<uint64_t> known[kMaxDevices];
  Launch l;
  const moe_status st = prepare_launch(kern, kThreads, smem, false, known, l);
  if (st != MOE_OK) return st;

  p.m_blocks = (p.N + BM - 1) / BM;
  const long used = p.rows < p.E ? p.rows : p.E;
  // tiles when all used groups are alike; few: narrower, then cut (gemm_grouped.cu)
  auto tiles_of = [&](long tile) {
    const long t = (p.rows + tile - 1) / tile;
    return (t > used ? t : used) * p.m_blocks;
  };
  p.tile = BT;
  while (p.tile > 64 && tiles_of(p.tile / 2) <= l.sms) p.tile /= 2;
  const int blocks = (p.K + BK - 1) / BK;
  p.split = 1;
  while (p.split < 8 && tiles_of(p.tile) * p.split * 2 <= l.sms && blocks >= 16 && blocks >= p.split * 8) p.split *= 2;
  const long tiles = ((long)(p.rows + p.tile - 1) / p.tile + used) * p.m_blocks;  // at most
  if (tiles > INT_MAX / 8) return MOE_ERR_UNSUPPORTED;
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.gridDim = dim3((unsigned)(p.split > 1 ? tiles * p.split : tiles < l.sms ? tiles : l.sms));
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = p.split > 1 ? 1 : 0;
  MOE_CUDA_TRY(cudaLaunchKernelEx(&lc, kern, ta, tb, tsa, tsb, p));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

moe_status launch_grouped_nvfp4(const MoEGrouped &g, const void *a, const void *sa, const float *ra,
                                const int32_t *offsets, const void *w, const void *sw, const float *rw,
                                const float *row_weight, void *y, int *status, cudaStream_t s) {
  Params p = {};
  p.rows = g.rows;
  p.N = g.n;
  p.K = g.k;
  p.E = g.groups;
  p.offsets = offsets;
  p.sa = (const uint8_t *)sa;
  p.sw = (const uint8_t *)sw;
  p.ra = ra;
  p.rw = rw;
  p.row_weight = row_weight;
  p.out = y;
  p.out_f32 = g.out_dtype == MOE_F32;
  p.status = status;
  // 64-token tiles and a deeper weight ring for few rows a group: 8 / 16 / 64 / 96
  // rows in each of 32 groups x 4096 x 2048: 35 / 35 / 39 / 50 us so, with tiles of
  // up to 192 tokens 37 / 37 / 39 / 41.  8192 rows over 128 groups: 113 us so and 119
  // with 192 when equal, 145 and 128 with sizes as 1 / i.
  const bool narrow = g.rows <= 64l * g.groups;
  const bool sf_tma = g.k % 256 == 0;
  if (narrow) return sf_tma ? launch<64, true>(p, a, w, s) : launch<64, false>(p, a, w, s);
  return sf_tma ? launch<192, true>(p, a, w, s) : launch<192, false>(p, a, w, s);
}

}  // namespace moe
