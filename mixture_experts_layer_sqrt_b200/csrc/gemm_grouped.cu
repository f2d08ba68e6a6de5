// Products grouped by expert with ragged group sizes, and their gradients, in
// bf16 on the 5th-generation tensor cores (tcgen05 + TMEM + TMA), fp32
// accumulation.  Group e owns the rows off[e] <= r < off[e+1] of A.
//
//   NT  y[r, :] = w_r * a[r, :] . W[e]^T        W [E, N, K]   (forward)
//   NN  y[r, :] = w_r * a[r, :] . W[e]          W [E, K, N]   (input gradient of a
//                                               product whose weights are [E, K, N])
//   TN  dW[e] (+)= sum_{r in e} dy[r, :]^T a[r, :]            (weight gradient)
//
// NT and NN put the weights on the MMA's M side and the tokens on its N side:
// a tile is 128 output features (a CTA pair: 256) x up to BT tokens of one
// group, and its MMAs run with N = the tile's tokens rounded up to 16 (32).  A
// ragged group therefore pads no MMA rows (with the tokens on the M side every
// group pads to 128), weights are read once per BT tokens, and for a handful of
// tokens the MMA is small and the kernel is a pure stream of the weights through
// the stage ring.  TN puts dy's features on M, a's on N and reduces over the
// group's rows; both operands are read as they lie (MN-major tiles), nothing is
// transposed in memory.
//
// Two shapes.  Up to 64 rows a group on average: single CTAs, 64-token tiles and
// eight 16 KB weight stages.  Above: 2-CTA pairs (cta_group::2) of 256 x 256
// tiles, each CTA with its own 128 features and half of the tokens.  A single
// CTA's 128 x 256 tile needs 96 bytes a cycle and SM from L2 at the MMAs' rate and
// got about 50; the pair needs 64 (512 rows a group x 4096 x 1536: 96 -> 87 us,
// tensor pipe 65 -> 80% of active cycles).
//
// Measured (B200, 1 kW limit; cool clocks / after a second of the same call):
//   16 rows x 4096 x 28672 over 8 groups      284 us = 6.6 TB/s, a copy's rate
//   15001 x 8192 x 2048 over 64 groups        504 / 610 us (cool: DRAM 5 TB/s and
//                                             1 PFLOP/s at once, 1.4 GHz)
//   65536 x 4096 x 1536 over 128 (NN)         661-810 / 883 us, tensor pipe 90%
//   8192 rows, dW 8 x 4096 x 14336 (TN)       679 / 795 us, tensor pipe 85%
// All of the last three are held by the power limit: the clock falls to 1.3-1.5
// GHz, and to 980, 990 and 1290 MHz after a while.  One cuBLAS product of their sizes
// (a single weight matrix) takes 338 / 398, 556 / 653 and 643 / 765 us.  Added to an
// existing dW the last takes 4.1 ms in fp32 and 2.9 in bf16 (see the epilogue's loop
// over the old values).
//
// A K-major tile lies in shared memory as rows of 64 reduction elements (128
// bytes, 128-byte swizzle); an MN-major tile as boxes of 64 features x 64
// reduction elements, a 128-byte line per reduction element.  The last block
// of a TN reduction brings in rows of the next group (or none): their lines
// are set to zero in both operands before the MMAs read them, so that nothing
// there, NaN included, reaches this group's sum.
//
// Roles (320 threads per CTA, 224 for TN; persistent, one CTA per SM):
//   warp 0    TMA producer into the stage ring
//   warp 1    TMEM owner; one thread issues the MMAs (4 x K=16 per stage);
//             two accumulators let the epilogue of tile i overlap the MMAs
//             of tile i+1
//   warps 2-9 epilogue: TMEM lane = output feature (TN: warps 2-5)
//   warp 6    TN: clears the lines above and hands the stage on to the MMAs
//
// Every wait is bounded (2 s, and 4 us for every stage that passes meanwhile; then
// MOE_ERR_DEVICE_TIMEOUT in the status word and an orderly wind down).
#include <cudaTypedefs.h>
#include <limits.h>

#include "grouped.cuh"
#include "kernels.h"
#include "tma_host.h"

namespace moe {

MOE_VIOLATION_COUNTER(violations_gemm_grouped)

namespace {

using namespace grouped;

enum Mode { NT = 0, NN = 1, TN = 2 };

constexpr int BM = 128;              // output features per tile (TMEM lanes)
constexpr int BK = 64;               // reduction elements per stage
constexpr int UMMA_K = 16;
constexpr int A_BYTES = BM * BK * 2;  // 16 KB
constexpr int BOX = 64 * BK * 2;     // 8 KB: an MN-major box

// BT: tokens (NT, NN) or columns (TN) per tile, the MMA's largest N.
// Pairs (BT = 256): a tile has 256 output features, 128 a CTA of a 2-CTA
// cluster; each CTA stages its own features and half of the tokens.
template <int BT>
struct Cfg {
  static constexpr bool PAIR = BT == 256;
  static constexpr int TILE_M = PAIR ? 2 * BM : BM;
  static constexpr int B_ROWS = PAIR ? BT / 2 : BT;  // staged by one CTA
  static constexpr int B_BYTES = B_ROWS * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = PAIR ? 6 : 8;
  static constexpr int TOK_BOX = PAIR ? 64 : 32;     // token rows per TMA box (NT, NN)
  static constexpr int N_STEP = PAIR ? 32 : 16;      // N of the MMAs is a multiple of it
  static constexpr uint32_t TMEM_COLS = 2 * BT;
};
template <Mode MODE>
constexpr int kEpiWarps = MODE == TN ? 4 : 4 * kEpiGroups;
template <Mode MODE>
constexpr int kThreads = MODE == TN ? 224 : 320;
constexpr int kClearWarp = 6;  // TN

template <int STAGES>
struct Smem {
  uint64_t full[STAGES];    // stage ready for the MMAs
  uint64_t landed[STAGES];  // TN: the copies of a last, partial block are complete in this CTA
  uint64_t empty[STAGES];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint64_t drain;
  __align__(16) float wbuf[4 * kEpiGroups * 32];  // row factors, 32 an epilogue warp
  uint32_t tmem_base;
  int abort;
  int start[MAX_E + 1];
  int off[MAX_E + 1];
};
constexpr int kSmemPart = 9728;             // barriers and tile list
constexpr int kStaging = 4 * 32 * 32 * 4;   // epilogue: 4 KB a warp (TN), or two buffers of 32 tokens
static_assert(kStaging == kRowStage, "one size for both epilogues");
static_assert(sizeof(Smem<8>) <= kSmemPart, "the epilogue staging follows the barriers and tile list");

struct Params {
  int rows, N, K, E;
  int m_blocks;    // TILE_M-feature blocks of the output
  int tile;        // tokens or columns of a tile, at most BT
  int n_blocks;    // TN: blocks of `tile` columns
  int split;       // parts that a tile's reduction is cut into, one a CTA (or pair) of a cluster
  const int32_t *offsets;
  const float *row_weight;
  void *out;       // y [rows, N] or dW [E, N, K]
  int out_f32;
  int accumulate;  // TN
  int *status;
};

// Both arrivals of a barrier that counts two, and the bytes to expect.
__device__ __forceinline__ void arrive2_expect_tx(uint64_t *bar, uint32_t bytes) {
  asm volatile(
      "mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n\t"
      "mbarrier.arrive.shared::cta.b64 _, [%0], 2;" ::"r"(ptx::smem_addr(bar)),
      "r"(bytes)
      : "memory");
}

__device__ __forceinline__ void spin_ns(uint64_t ns) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (ptx::globaltimer_ns() - t0 < ns) {
  }
}

// Shared-memory descriptor of an MN-major tile with the 128-byte swizzle:
// boxes of 64 features (128 bytes) x 64 reduction elements; leading byte
// offset = next 64 features (one box), stride byte offset = next 8 reduction
// elements (1024 bytes).
__device__ __forceinline__ uint64_t desc_mnmajor_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(BOX >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

template <Mode MODE, int BT>
__global__ void __launch_bounds__(kThreads<MODE>, 1)
    grouped_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Params p) {
  using C = Cfg<BT>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *stage_a = base;
  uint8_t *stage_b = base + STAGES * A_BYTES;
  Smem<STAGES> &sm = *reinterpret_cast<Smem<STAGES> *>(base + STAGES * C::STAGE_BYTES);
  uint32_t *staging = reinterpret_cast<uint32_t *>(base + STAGES * C::STAGE_BYTES + kSmemPart);

  constexpr bool PAIR = C::PAIR;

  // split: this CTA's partial sums, over the stage buffers once the MMAs have read them
  float *parts = reinterpret_cast<float *>(base);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a cluster: `split` CTAs or pairs, which share a tile
  const uint32_t crank = ptx::cluster_ctarank();
  const uint32_t rank = PAIR ? crank & 1u : 0u;     // in the pair
  const uint32_t lead = crank - rank;               // the pair's leader
  const int part = PAIR ? (int)(crank >> 1) : (int)crank;
  const int csize = PAIR ? 2 * p.split : p.split;
  const int unit = (int)blockIdx.x / csize, n_units = (int)gridDim.x / csize;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(&sm.full[s], MODE == TN ? 2 : 1);  // TN: a partial block is handed on by both CTAs
      ptx::mbar_init(&sm.landed[s], 1);
      ptx::mbar_init(&sm.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&sm.tmem_full[a], 1);
      ptx::mbar_init(&sm.tmem_empty[a], (PAIR ? 2 : 1) * kEpiWarps<MODE>);
    }
    ptx::mbar_init(&sm.drain, 1);
    sm.abort = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    if (PAIR) {
      ptx::tmem_alloc_pair(&sm.tmem_base, C::TMEM_COLS);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(&sm.tmem_base, C::TMEM_COLS);
      ptx::tmem_relinquish();
    }
  }
  load_offsets(p.offsets, p.rows, p.E, sm.off);
  __syncthreads();
  if (warp == 2 && (MODE != TN || kChecked)) {
    // TN needs no tile list (every group has m_blocks * n_blocks tiles), but
    // the same check of the offsets
    const bool ok = scan_tiles(sm.off, p.E, p.rows, p.tile, sm.start);
    if (kChecked && !ok && lane == 0 && blockIdx.x == 0) note_violation();
    if (kChecked && MODE == TN && lane == 0) sm.start[0] = ok ? 0 : 1;
  }
  ptx::tc_fence_before();
  __syncwarp();
  if (PAIR) ptx::cluster_sync();  // the peer's copies and arrivals may reach this CTA's barriers from here on
  else __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = sm.tmem_base;
  int total;
  if (MODE == TN) total = (kChecked && sm.start[0]) ? 0 : p.E * p.m_blocks * p.n_blocks;
  else total = sm.start[p.E] * p.m_blocks;

  // tile t -> group, feature block, first row / column, reduction blocks
  struct Tile {
    int e, m0, c0, count, row0;  // c0: first column (TN); count: tokens or columns; row0: first token
    int k0, red;                 // this part's first reduction element (TN: row) and their number
    int blocks;                  // reduction blocks of all parts
    __device__ int first_block(int part, int split) const { return (int)((long)blocks * part / split); }
    // MMA N, and the tokens or columns that this CTA stages of it
    __device__ int width() const { return (count + C::N_STEP - 1) & ~(C::N_STEP - 1); }
    __device__ int staged() const { return PAIR ? width() / 2 : width(); }
  };
  auto tile_of = [&](int t) {
    Tile r;
    if (MODE == TN) {
      const int per = p.m_blocks * p.n_blocks;
      r.e = t / per;
      const int local = t - r.e * per;
      const int nb = local / p.m_blocks;
      r.m0 = (local - nb * p.m_blocks) * C::TILE_M;
      r.c0 = nb * p.tile;
      r.count = p.K - r.c0 < p.tile ? p.K - r.c0 : p.tile;
      r.row0 = 0;
      r.k0 = sm.off[r.e];
      r.red = group_rows(sm.off, r.e);
    } else {
      const TokenTile tt = token_tile(sm.start, sm.off, p.E, p.m_blocks, t, C::N_STEP);
      r.e = tt.e;
      r.m0 = tt.blk * C::TILE_M;
      r.c0 = 0;
      r.row0 = tt.row0;
      r.count = tt.count;
      r.k0 = 0;
      r.red = p.K;
    }
    r.blocks = (r.red + BK - 1) / BK;
    if (p.split > 1) {
      const int b0 = r.first_block(part, p.split), b1 = r.first_block(part + 1, p.split);
      r.k0 += b0 * BK;
      r.red = (b1 * BK < r.red ? b1 * BK : r.red) - b0 * BK;
      if (r.red < 0) r.red = 0;
    }
    return r;
  };

  if (warp == 0) {
    // ================================================= TMA producer
    if (elect_one()) {
      uint32_t used = 0, phase = 0;  // TN: stages whose landed barrier was used, and its next phase
      Ring<STAGES> ring;
      uint32_t issued = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += n_units) {
        const Tile tl = tile_of(t);
        const int kbs = (tl.red + BK - 1) / BK;
        const int staged = tl.staged();
        const int boxes = MODE == TN ? (staged + 63) / 64 : (staged + C::TOK_BOX - 1) / C::TOK_BOX;
        const uint32_t tx = A_BYTES + (uint32_t)boxes * (MODE == TN ? BOX : C::TOK_BOX * BK * 2);
        const int m0 = tl.m0 + (int)rank * BM;                                    // this CTA's features
        const int b0 = (MODE == TN ? tl.c0 : tl.row0) + (int)rank * staged;       // and columns or tokens
        for (int kb = 0; kb < kbs; ++kb, ring.next(), ++issued) {
          if (!wait_bar(&sm.empty[ring.s], ring.ph ^ 1u, &sm.abort, p.status)) {
            ok = false;
            break;
          }
          uint64_t *bar = &sm.full[ring.s];
          uint8_t *a = stage_a + ring.s * A_BYTES;
          uint8_t *b = stage_b + ring.s * C::B_BYTES;
          const int k0 = tl.k0 + kb * BK;
          const bool partial = MODE == TN && tl.red - kb * BK < BK;
          if (PAIR && !partial) {
            // both CTAs' copies complete on the leader's barrier
            const uint32_t lead_bar = ptx::map_to_rank(bar, lead);
            if (rank == 0) {
              if (MODE == TN) arrive2_expect_tx(bar, 2 * tx);
              else ptx::mbar_arrive_expect_tx(bar, 2 * tx);
            }
            if (MODE == NT) {
              ptx::tma_load_3d_pair(a, &tmA, lead_bar, k0, m0, tl.e);
            } else if (MODE == NN) {
              ptx::tma_load_3d_pair(a, &tmA, lead_bar, m0, k0, tl.e);
              ptx::tma_load_3d_pair(a + BOX, &tmA, lead_bar, m0 + 64, k0, tl.e);
            } else {
              ptx::tma_load_2d_pair(a, &tmA, lead_bar, m0, k0);
              ptx::tma_load_2d_pair(a + BOX, &tmA, lead_bar, m0 + 64, k0);
            }
            for (int i = 0; i < boxes; ++i) {
              if (MODE == TN) ptx::tma_load_2d_pair(b + i * BOX, &tmB, lead_bar, b0 + i * 64, k0);
              else ptx::tma_load_2d_pair(b + i * C::TOK_BOX * BK * 2, &tmB, lead_bar, k0, b0 + i * C::TOK_BOX);
            }
            continue;
          }
          if (MODE == TN) {  // the clearing warp hands the stage on
            bar = &sm.landed[ring.s];
            used |= 1u << ring.s;
            phase ^= 1u << ring.s;
          }
          ptx::mbar_arrive_expect_tx(bar, tx);
          if (MODE == NT) {
            ptx::tma_load_3d(a, &tmA, bar, k0, m0, tl.e);
          } else if (MODE == NN) {
            ptx::tma_load_3d(a, &tmA, bar, m0, k0, tl.e);
            ptx::tma_load_3d(a + BOX, &tmA, bar, m0 + 64, k0, tl.e);
          } else {
            ptx::tma_load_2d(a, &tmA, bar, m0, k0);
            ptx::tma_load_2d(a + BOX, &tmA, bar, m0 + 64, k0);
          }
          for (int i = 0; i < boxes; ++i) {
            if (MODE == TN) ptx::tma_load_2d(b + i * BOX, &tmB, bar, b0 + i * 64, k0);
            else ptx::tma_load_2d(b + i * C::TOK_BOX * BK * 2, &tmB, bar, k0, b0 + i * C::TOK_BOX);
          }
        }
      }
      // every issued copy has landed before shared memory is released (a peer's
      // complete on the leader's barriers, which the leader waits for)
      for (int s = 0; s < STAGES; ++s) {
        if (MODE == TN && (used >> s & 1)) drain_bar(&sm.landed[s], (phase >> s & 1) ^ 1u, p.status);
        if (rank != 0 || (uint32_t)s >= issued) continue;
        const uint32_t last = (issued - 1 - s) / STAGES;  // this stage's last round
        drain_bar(&sm.full[s], last & 1u, p.status);
      }
      if (rank != 0 && !ok) spin_ns(1000000);  // an aborting peer gives its last copies time to land
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================================================= MMA issuer (a pair's leader)
    if (rank == 0 && elect_one()) {
      // D fp32, A and B bf16; bit 15: A is MN-major, bit 16: B is
      constexpr uint32_t idesc0 =
          ptx::idesc_bf16_f32(C::TILE_M, 0) | (MODE != NT ? 1u << 15 : 0u) | (MODE == TN ? 1u << 16 : 0u);
      // descriptors of stage 0; an address moves by its bytes >> 4
      const uint64_t ad0 = MODE == NT ? ptx::desc_kmajor_sw128(ptx::smem_addr(stage_a))
                                      : desc_mnmajor_sw128(ptx::smem_addr(stage_a));
      const uint64_t bd0 = MODE == TN ? desc_mnmajor_sw128(ptx::smem_addr(stage_b))
                                      : ptx::desc_kmajor_sw128(ptx::smem_addr(stage_b));
      constexpr uint32_t a_step = (MODE == NT ? UMMA_K * 2 : UMMA_K * 128) >> 4;
      constexpr uint32_t b_step = (MODE == TN ? UMMA_K * 128 : UMMA_K * 2) >> 4;
      auto mma = [](uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
        if (PAIR) ptx::mma_bf16_pair(d, a, b, id, acc);
        else ptx::mma_bf16(d, a, b, id, acc);
      };
      const uint16_t both = (uint16_t)(0x3u << lead);
      auto commit = [both](uint64_t *bar) {  // pairs: on both CTAs' barriers
        if (PAIR) ptx::mma_commit_pair_mc(bar, both);
        else ptx::mma_commit(bar);
      };
      Ring<STAGES> ring;
      bool ready = false;  // the next stage's barrier, read ahead of the MMAs before it
      int i = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += n_units) {
        const Tile tl = tile_of(t);
        const int kbs = (tl.red + BK - 1) / BK;
        if (kbs == 0) continue;  // TN, empty group: the epilogue needs no sum
        const int acc = i & 1;
        const uint32_t aph = (i >> 1) & 1u;
        ++i;
        if (!wait_bar(&sm.tmem_empty[acc], aph ^ 1u, &sm.abort, p.status)) break;
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BT;
        const uint32_t idesc = idesc0 | (uint32_t)(tl.width() >> 3) << 17;
        for (int kb = 0; kb < kbs; ++kb) {
          if (!ready && !wait_bar(&sm.full[ring.s], ring.ph, &sm.abort, p.status)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          Ring<STAGES> nx = ring;
          nx.next();
          ready = ptx::mbar_try_wait(&sm.full[nx.s], nx.ph);
          const uint64_t ad = ad0 + (uint32_t)ring.s * (A_BYTES >> 4), bd = bd0 + (uint32_t)ring.s * (C::B_BYTES >> 4);
          const int left = tl.red - kb * BK;
          if (MODE == TN && left <= BK - UMMA_K) {
            const int steps = (left + UMMA_K - 1) / UMMA_K;
            for (int k = 0; k < steps; ++k)
              mma(d_tmem, ad + k * a_step, bd + k * b_step, idesc, (kb | k) != 0);
          } else {
#pragma unroll
            for (int k = 0; k < BK / UMMA_K; ++k)
              mma(d_tmem, ad + k * a_step, bd + k * b_step, idesc, (kb | k) != 0);
          }
          commit(&sm.empty[ring.s]);
          ring = nx;
        }
        if (ok) commit(&sm.tmem_full[acc]);
      }
      // all issued MMAs complete before TMEM is released
      if (PAIR) ptx::mma_commit_pair(&sm.drain);
      else ptx::mma_commit(&sm.drain);
      drain_bar(&sm.drain, 0, p.status);
    }
    __syncwarp();
  } else if (MODE == TN && warp == kClearWarp) {
    // ================================================= lines of other rows (TN)
    uint32_t at = 0, phase = 0;  // blocks so far; next phase of each stage's landed barrier
    uint32_t since = 0;          // blocks and epilogues (as 16 blocks) since the last partial block
    for (int t = unit; t < total; t += n_units) {
      const Tile tl = tile_of(t);
      const int left = tl.red % BK;
      at += (tl.red + BK - 1) / BK;
      since += (tl.red + BK - 1) / BK + 16;
      if (left == 0) continue;
      const int s = (at - 1) % STAGES;
      if (!warp_wait(&sm.landed[s], phase >> s & 1, &sm.abort, p.status, since)) break;
      since = 0;
      __syncwarp();
      // lines [left, the MMAs' last) of every box
      uint8_t *a = stage_a + s * A_BYTES + left * 128, *b = stage_b + s * C::B_BYTES + left * 128;
      const int boxes = (tl.staged() + 63) / 64;
      const int pieces = (((left + UMMA_K - 1) & ~(UMMA_K - 1)) - left) * 8;  // of 16 bytes, a box
      for (int j = lane; j < pieces; j += 32) {
#pragma unroll
        for (int i = 0; i < 2 + C::B_ROWS / 64; ++i)
          if (i < 2 + boxes)
            *reinterpret_cast<uint4 *>((i < 2 ? a + i * BOX : b + (i - 2) * BOX) + j * 16) = make_uint4(0, 0, 0, 0);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (rank != 0) ptx::mbar_arrive_cluster(ptx::map_to_rank(&sm.full[s], lead));
        else ptx::mbar_arrive(&sm.full[s]);
      }
      phase ^= 1u << s;
    }
  } else {
    // ================================================= epilogue (from warp 2 on)
    const int q = warp & 3;              // TMEM lane quadrant this warp may access
    const int group = (warp - 2) >> 2;   // NT, NN
    const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
    const RowStore store = {p.out, p.out_f32, p.N, p.row_weight, nullptr};
    int i = 0;
    for (int t = unit; t < total; t += n_units) {
      const Tile tl = tile_of(t);
      const bool have = tl.red > 0;
      const int acc = i & 1;
      const uint32_t aph = (i >> 1) & 1u;
      const float w0 = MODE != TN ? row_factor(store, tl.row0, tl.count, group * 32) : 1.0f;
      if (have) {
        ++i;
        if (!all_agree<3, 32 * kEpiWarps<MODE>>(
                warp_wait(&sm.tmem_full[acc], aph, &sm.abort, p.status, (tl.red + BK - 1) / BK)))
          break;
        ptx::tc_fence_after();
      }
      const uint32_t tbase = tmem_base + lane_addr + acc * BT;
      if (p.split > 1) {
        if (!have) {
        } else if (MODE != TN) {
          put_part_columns(parts, tbase, tl.count, q, group, kEpiGroups);
        } else {
          put_part_features(parts, tbase, tl.count, p.tile + 4, q);
        }
      } else if (MODE != TN) {
        store_tokens<false>(store, tbase, tl.row0, tl.count, tl.m0 + (int)rank * BM, q, group, w0, 1.0f,
                            reinterpret_cast<uint8_t *>(staging), sm.wbuf + (warp - 2) * 32);
      } else {
        // rows of dW, a lane each: 32 words of every row at a time through this
        // warp's 4 KB (16-byte piece j of row r at j ^ (r % 8)), so that every
        // store writes four whole 128-byte row segments
        uint32_t *stg = staging + q * 32 * 32;
        const int n_first = tl.m0 + (int)rank * BM + q * 32;
        const int rr = lane >> 3, ff = lane & 7;
        const bool fp32 = p.out_f32 || p.accumulate;  // words: fp32 sums, or bf16 pairs rounded here
        if (!fp32) {
          uint32_t lo[32], hi[32];
          if (have) {
            ptx::tmem_ld32(tbase, lo);
            ptx::tmem_ld32(tbase + 32, hi);
          }
#pragma unroll 1
          for (int c = 0; c < tl.count; c += 64) {
            uint4 val[8];
            if (have) {
              ptx::tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int i = 8 * (j & 3) + 2 * k;
                  const __nv_bfloat162 o =
                      j < 4 ? __floats2bfloat162_rn(__uint_as_float(lo[i]), __uint_as_float(lo[i + 1]))
                            : __floats2bfloat162_rn(__uint_as_float(hi[i]), __uint_as_float(hi[i + 1]));
                  w[k] = *reinterpret_cast<const uint32_t *>(&o);
                }
                *reinterpret_cast<uint4 *>(stg + lane * 32 + ((j ^ (lane & 7)) << 2)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
              }
              if (c + 64 < tl.count) {
                ptx::tmem_ld32(tbase + c + 64, lo);
                ptx::tmem_ld32(tbase + c + 96, hi);
              }
              __syncwarp();
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int r = 4 * k + rr;
                val[k] = *reinterpret_cast<const uint4 *>(stg + r * 32 + ((ff ^ (r & 7)) << 2));
              }
              __syncwarp();
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k) val[k] = make_uint4(0, 0, 0, 0);
            }
            const int col = tl.c0 + c + ff * 8;
            __nv_bfloat16 *dst = (__nv_bfloat16 *)p.out + ((long)tl.e * p.N + n_first + rr) * p.K + col;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (n_first + 4 * k + rr < p.N && col < p.K) *reinterpret_cast<uint4 *>(dst + (long)(4 * k) * p.K) = val[k];
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < tl.count; c += 32) {
            float4 val[8];
            if (have) {
              uint32_t v[32];
              ptx::tmem_ld32(tbase + c, v);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4 *>(stg + lane * 32 + ((j ^ (lane & 7)) << 2)) =
                    make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
              __syncwarp();
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int r = 4 * k + rr;
                val[k] = *reinterpret_cast<const float4 *>(stg + r * 32 + ((ff ^ (r & 7)) << 2));
              }
              __syncwarp();
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k) val[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            const int col = tl.c0 + c + ff * 4;
            const long at = ((long)tl.e * p.N + n_first + rr) * p.K + col;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (n_first + 4 * k + rr >= p.N || col >= p.K || (!have && p.accumulate)) continue;
              float4 x = val[k];
              if (p.out_f32) {
                float4 *dst = reinterpret_cast<float4 *>((float *)p.out + at + (long)(4 * k) * p.K);
                if (p.accumulate) {
                  const float4 old = *dst;
                  x = make_float4(old.x + x.x, old.y + x.y, old.z + x.z, old.w + x.w);
                }
                *dst = x;
              } else {  // added in fp32, rounded once
                uint2 *dst = reinterpret_cast<uint2 *>((__nv_bfloat16 *)p.out + at + (long)(4 * k) * p.K);
                const uint2 old = *dst;
                const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&old.x));
                const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&old.y));
                const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x + x.x, a.y + x.y);
                const __nv_bfloat162 hi = __floats2bfloat162_rn(b.x + x.z, b.y + x.w);
                *dst = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
              }
            }
          }
        }
      }
      if (have) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) arrive_cluster_relaxed(ptx::map_to_rank(&sm.tmem_empty[acc], lead));
          else ptx::mbar_arrive(&sm.tmem_empty[acc]);
        }
      }
    }
  }

  if (p.split > 1) {
    // the parts' sums, in the parts' order, each part a share of the columns
    __syncwarp();
    ptx::cluster_sync();
    if (unit < total) {
      const Tile tl = tile_of(unit);
      const int n0 = tl.m0 + (int)rank * BM;
      uint32_t has = 0;  // parts with something to add
      for (int k = 0; k < p.split; ++k)
        if (tl.first_block(k, p.split) < tl.first_block(k + 1, p.split)) has |= 1u << k;
      constexpr uint32_t step = PAIR ? 2 : 1;
      if (MODE != TN) {
        const int c_lo = tl.count * part / p.split, w = tl.count * (part + 1) / p.split - c_lo;
        const RowStore store = {p.out, p.out_f32, p.N, p.row_weight, nullptr};
        store_summed_tokens(store, parts, tl.row0, c_lo, w, n0, nullptr, rank, step, p.split, has, kThreads<MODE>);
      } else if (has || !p.accumulate) {
        constexpr int U = 4;
        const int quads = tl.count / 4;                                      // of a row
        const int f_lo = BM * part / p.split, rows = BM / p.split;            // split: a power of two
        const int all = rows * quads;
        for (int i0 = threadIdx.x; i0 < all; i0 += U * kThreads<MODE>) {
          int at[U];
          float4 sum[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int i = min(i0 + u * kThreads<MODE>, all - 1), f = i / quads;
            at[u] = (f_lo + f) * (p.tile + 4) + (i - f * quads) * 4;
          }
          add_parts(parts, at, rank, step, p.split, has, sum);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kThreads<MODE>, f = i / quads, n = n0 + f_lo + f;
            if (i < all && n < p.N)
              put_quad(p.out, p.out_f32, ((long)tl.e * p.N + n) * p.K + tl.c0 + (i - f * quads) * 4, sum[u],
                       p.accumulate != 0);
          }
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncwarp();
  if (csize > 1) ptx::cluster_sync();  // neither CTA leaves while the pair's copies, MMAs or arrivals are pending
  else __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    if (PAIR) ptx::tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else ptx::tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <Mode MODE, int BT>
moe_status launch(Params &p, const void *a, const void *b, cudaStream_t s) {
  using C = Cfg<BT>;
  CUtensorMap ta, tb;
  bool ok;
  if (MODE == NT) {
    ok = tma_map_bf16(&ta, a, 3, (uint64_t)p.K, (uint64_t)p.N, (uint64_t)p.E, BM) &&
         tma_map_bf16(&tb, b, 2, (uint64_t)p.K, (uint64_t)p.rows, 1, C::TOK_BOX);
  } else if (MODE == NN) {
    ok = tma_map_bf16(&ta, a, 3, (uint64_t)p.N, (uint64_t)p.K, (uint64_t)p.E, BK) &&
         tma_map_bf16(&tb, b, 2, (uint64_t)p.K, (uint64_t)p.rows, 1, C::TOK_BOX);
  } else {
    ok = tma_map_bf16(&ta, a, 2, (uint64_t)p.N, (uint64_t)p.rows, 1, BK) &&
         tma_map_bf16(&tb, b, 2, (uint64_t)p.K, (uint64_t)p.rows, 1, BK);
  }
  if (!ok) return MOE_ERR_CUDA;
  const size_t smem = 1024 + (size_t)C::STAGES * C::STAGE_BYTES + kSmemPart + kStaging;
  auto kern = grouped_gemm<MODE, BT>;
  static std::atomic<uint64_t> known[kMaxDevices];
  Launch l;
  const moe_status st = prepare_launch(kern, kThreads<MODE>, smem, C::PAIR, known, l);
  if (st != MOE_OK) return st;

  p.m_blocks = (p.N + C::TILE_M - 1) / C::TILE_M;
  const long used = p.rows < p.E ? p.rows : p.E;  // groups that can have rows
  const long units = C::PAIR ? l.pairs : l.sms;
  // tiles when all used groups are alike
  auto tiles_of = [&](long tile) {
    if (MODE == TN) return (long)p.E * p.m_blocks * ((p.K + tile - 1) / tile);
    const long t = (p.rows + tile - 1) / tile;
    return (t > used ? t : used) * p.m_blocks;
  };
  // Few tiles: narrower ones, then the reduction cut into parts, as long as they
  // all run at once.  A block takes about 0.2 us when few CTAs run, the cluster
  // and its sum 2.5 us (200 rows x 512 x 128: 5.9 us whole, 8.4 in two parts;
  // 1 row x 14336 x 4096: 49 us whole, 28 in four): cut from 32 blocks on, into
  // parts of at least eight.
  p.tile = BT;
  while (p.tile > 64 && tiles_of(p.tile / 2) <= units) p.tile /= 2;
  const long blocks = ((MODE == TN ? p.rows / used : p.K) + BK - 1) / BK;
  const int most = C::PAIR ? 4 : 8;  // CTAs of a cluster: 8
  p.split = 1;
  while (p.split < most && tiles_of(p.tile) * p.split * 2 <= units && blocks >= 32 && blocks >= p.split * 16) p.split *= 2;
  p.n_blocks = (p.K + p.tile - 1) / p.tile;
  const long tiles =
      MODE == TN ? tiles_of(p.tile) : ((long)(p.rows + p.tile - 1) / p.tile + used) * p.m_blocks;  // at most
  if (tiles > INT_MAX / 8) return MOE_ERR_UNSUPPORTED;
  const int csize = (C::PAIR ? 2 : 1) * p.split;
  // split: a cluster a tile; else every CTA or pair that fits walks the tiles
  const long grid = p.split > 1 ? tiles * csize : (tiles < units ? tiles : units) * csize;
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)csize;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.gridDim = dim3((unsigned)grid);
  lc.blockDim = dim3(kThreads<MODE>);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = csize > 1 ? 1 : 0;
  MOE_CUDA_TRY(cudaLaunchKernelEx(&lc, kern, ta, tb, p));
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace

moe_status launch_grouped_bf16(const MoEGrouped &g, const void *a, const int32_t *offsets, const void *w,
                               bool transposed, const float *row_weight, void *y, int *status, cudaStream_t s) {
  Params p = {};
  p.rows = g.rows;
  p.N = g.n;
  p.K = g.k;
  p.E = g.groups;
  p.offsets = offsets;
  p.row_weight = row_weight;
  p.out = y;
  p.out_f32 = g.out_dtype == MOE_F32;
  p.status = status;
  // few rows a group: single CTAs with narrow token tiles.  8 / 16 / 64 / 96 / 128
  // rows in each of 32 groups x 4096 x 2048: 91 / 92 / 96 / 112 / 114 us so, with
  // pairs 96 / 97 / 102 / 104 / 106.  The host knows the average only: 8192 rows over
  // 128 groups take 346 us so and 359 with pairs when equal, 407 and 368 with sizes
  // as 1 / i.
  const bool narrow = g.rows <= 64l * g.groups;
  if (transposed) return narrow ? launch<NN, 64>(p, w, a, s) : launch<NN, 256>(p, w, a, s);
  return narrow ? launch<NT, 64>(p, w, a, s) : launch<NT, 256>(p, w, a, s);
}

moe_status launch_grouped_wgrad_bf16(const MoEGrouped &g, const void *dy, const void *a, const int32_t *offsets,
                                     bool accumulate, void *dw, int *status, cudaStream_t s) {
  Params p = {};
  p.rows = g.rows;
  p.N = g.n;
  p.K = g.k;
  p.E = g.groups;
  p.offsets = offsets;
  p.out = dw;
  p.out_f32 = g.out_dtype == MOE_F32;
  p.accumulate = accumulate;
  p.status = status;
  return launch<TN, 256>(p, dy, a, s);
}

}  // namespace moe
