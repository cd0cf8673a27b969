// 16-bit (BF16 / FP16) matrix products with FP32 accumulation on the 5th-generation tensor
// cores: grouped by expert with ragged row segments, or dense with a bias, activation and
// residual epilogue, and the products of their backward passes.
//
//   forward  y[i]  = x[i] W_e^T            dense: z = x W^T + b, y = act(z) + residual
//   dgrad    dx[i] = dy[i] W_e
//   wgrad    dW_e  = sum_i dy[i]^T x[i]    over the rows i of expert e's segment
//
// One kernel computes D[i][j] = sum_r A[i][r] B[j][r] for all three; an operand whose r runs
// along memory is K-major in shared memory, one whose i or j does is MN-major (the transposed
// read is the tensor core's: no operand is ever transposed in memory).
//
// A pair of CTAs (one on each SM of a TPC) computes a tile of up to 256 x 256: each loads its half
// of A's and of B's rows (32 KB per 64-deep step, 5 stages; 6 measured the same, 4 4 % slower at
// 4096 x 5120 x 5120), tcgen05.mma.cta_group::2 reads both halves of B from both shared memories,
// and each CTA holds its 128 x 256 FP32 accumulator in tensor memory, double buffered, so the
// epilogue of one tile overlaps the next one's MMAs.  In forward and dgrad the 256 features of the
// weights are the instruction's M side and the token rows its N side: N follows a segment's last rows
// in steps of 32, so a ragged segment costs tensor time for its own rows only.
//
// Per CTA: warp 0 loads (TMA, 128-byte swizzle), both CTAs' bytes counted on the first CTA's
// barrier; warp 1 of the first CTA issues the MMAs; warps 4-11 run the epilogue: forward and dgrad
// transpose 32 x 32 pieces through shared memory, stored by TMA from there (a segment's last rows, which no
// map can clip, row by row); wgrad, whose rows are never ragged, in 128-byte x 32-row pieces (an expert's few rows make
// few steps a tile, so its output counts most: 64 experts of 128 rows, 5120 x 2560, 468 us, with plain stores
// 931 us; its 1678 MB alone are a fill of 228 us).
//
// Ragged ends.  In forward and dgrad, rows behind a segment's end only feed accumulator columns that
// are not stored.  In wgrad the reduction runs over rows, so the last step of a segment would add
// rows of the next one (or rows never written, where a NaN passes even a zero factor): each
// segment has tensor maps of its own, built on the device from the offsets, whose row bound makes
// the loads fill zeros behind its end (and read nothing there: see launch_mm_table).  (Zeroing those lines in
// shared memory before the MMAs cost every tile a cross-CTA fence: 64 skewed experts, 32768 rows, 1011 us.)
//
// Every wait is bounded; one that runs out raises the timeout bit of the status word and the abort flag of
// every CTA of its cluster, which wind down together.
//
// Measured in a replayed graph, and called for long (at the power cap): 4096 x 5120 x 5120 150 us (1.43 PFLOP/s); 4096 x
// 20480, K = 5120 with GELU and saved sums 587 to 602 us (by card) and 693 to 731; 64 skewed experts, 32768 rows,
// 2560 -> 5120 704 to 757 and 845 to 920; both gradients of 32 experts, 8192 rows, 470 to 483 and 564 to 578; 32 rows
// over 64 experts, 5120 -> 2560, 111 (6.4 TB/s) and 113.
#include "common.cuh"
#include "dense.h"
#include "dense_epilogue.cuh"
#include "kernels.h"

namespace nvfp4moe {

namespace {

constexpr int kBK = 64;                  // reduction values per stage (one 128-byte swizzle row)
constexpr int kPairTile = 256;           // rows and columns of a pair's tile
constexpr int kHalf = 128;               // each CTA's share of A rows and of B rows
constexpr int kPairStages = 5;
constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 128 + 32 * kPairEpiWarps;
constexpr int kOperandBytes = kHalf * kBK * 2;
constexpr int kRasterRows = 16;          // row tiles that share a column tile before the next one

// ------------------------------------------------------------- cluster helpers ----
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Shared-memory address of this CTA -> the same address in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Arrival on CTA `rank`'s barrier; the release form also makes this thread's earlier
// shared-memory writes visible across the cluster.
__device__ __forceinline__ void mbar_arrive_rank(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(map_rank(smem_u32(bar), rank)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_rank_release(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_rank(smem_u32(bar), rank))
               : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait with cluster-scope acquire, ended early by the CTA's abort flag.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, const int* abort_flag,
                                             uint64_t limit_ns) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  uint32_t n = 0;
  while (!mbar_try_wait_cluster(bar, parity)) {
    if ((++n & 63u) == 0u &&
        (*reinterpret_cast<const volatile int*>(abort_flag) != 0 || globaltimer_ns() - t0 > limit_ns))
      return false;
  }
  return true;
}

// Stores v at this CTA's address `dst` in CTA `rank` and counts the 4 bytes on that CTA's barrier.
__device__ __forceinline__ void store_rank(int* dst, uint64_t* bar, uint32_t rank, int v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(
                   map_rank(smem_u32(dst), rank)),
               "r"(v), "r"(map_rank(smem_u32(bar), rank))
               : "memory");
}

__device__ __forceinline__ void set_abort(int* flag, uint32_t* status) {
  raise_status(status, kStatusTimeout);
  *reinterpret_cast<volatile int*>(flag) = 1;
}

// Before a warp's last barrier of the cluster: a CTA that gave up ends the waits of its cluster's others too (they are
// there until that barrier).  Done here once, not where a wait runs out: in every such place it was code enough
// to cost short calls their instruction fetches (both gradients of 13 experts, 1531 rows, 520 x 776: 33.4 us, here 32.4).
__device__ __forceinline__ void spread_abort(int* flag, int ctas) {
  if (*reinterpret_cast<volatile int*>(flag) == 0) return;
  for (int r = 0; r < ctas; ++r)
    asm volatile("st.relaxed.cluster.shared::cluster.b32 [%0], %1;" ::"r"(map_rank(smem_u32(flag), (uint32_t)r)), "r"(1)
                 : "memory");
}

// Tiled load into this CTA's shared memory, completion counted on a barrier of either CTA of the
// pair (bar: a shared::cluster address).
__device__ __forceinline__ void tma_load_pair(void* dst, const void* tmap, uint32_t bar, int32_t c0, int32_t c1,
                                              int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Makes a tensor map written by an earlier kernel usable by this thread's copies.
__device__ __forceinline__ void acquire_tmap(const void* tmap) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(tmap) : "memory");
}

// ------------------------------------------------------------ tcgen05, CTA pairs ----
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Arrives on `bar` of both CTAs of the pair when this thread's tcgen05 operations so far are done.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// The same on this CTA's `bar` alone.
__device__ __forceinline__ void tc_commit_pair_local(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// MN-major operand, 128-byte swizzle: 64 consecutive i (or j) per 128-byte line, one line per r;
// 8 lines form a 1024-byte group, groups 1024 bytes apart along r; blocks of 64 i are
// `block_bytes` apart.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t block_bytes) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(block_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Instruction descriptor of kind::f16: FP32 accumulator, A and B of one 16-bit type, their
// majorness, N / 8 at bit 17, M / 16 at bit 24.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t m, uint32_t n, bool fp16, bool a_mn, bool b_mn) {
  return (1u << 4) | ((fp16 ? 0u : 1u) << 7) | ((fp16 ? 0u : 1u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// --------------------------------------------------------------------- tiles ----
struct Tile {
  int e;
  int a0, b0;        // kMmWgrad: first i, first j; else first token row, first j
  int64_t out_row;   // row of D (in the whole output) that a0 is
  int rows_valid;    // rows of the tile to store
  int out_e;         // matrix of the output (or of its parts) that the tile belongs to
  int k0, steps;     // first 64-deep reduction step and how many
};

template <int kMode>
__device__ __forceinline__ int total_tiles(const MmArgs& p, int tile_i, int tile_j) {
  const int ntj = (p.J + tile_j - 1) / tile_j;
  if constexpr (kMode == kMmWgrad) return p.split * p.E * ((p.I + tile_i - 1) / tile_i) * ntj;
  return (p.tiles != nullptr ? p.tiles[p.E] : p.split * (int)((p.rows + tile_i - 1) / tile_i)) * ntj;
}

// Tile w in expert-major order; within an expert, blocks of kRasterRows row tiles go through the
// column tiles together, row tile fastest (a column tile's weights are read by its row tiles at
// about the same time, and a block's rows stay in L2 while it goes through the columns).
template <int kMode>
__device__ __forceinline__ Tile tile_at(const MmArgs& p, int w, int tile_i, int tile_j) {
  Tile t;
  const int ntj = (p.J + tile_j - 1) / tile_j;
  int mt_e, local, seg_row = 0, part = 0;
  int64_t seg_rows = p.rows;
  if constexpr (kMode == kMmWgrad) {
    mt_e = (p.I + tile_i - 1) / tile_i;
    t.out_e = w / (mt_e * ntj);
    local = w - t.out_e * mt_e * ntj;
    part = t.out_e / p.E;
    t.e = t.out_e - part * p.E;
  } else if (p.tiles != nullptr) {
    int lo = 0, hi = p.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.tiles[mid] * ntj <= w) lo = mid; else hi = mid;
    }
    t.e = lo;
    t.out_e = 0;
    mt_e = p.tiles[lo + 1] - p.tiles[lo];
    local = w - p.tiles[lo] * ntj;
  } else {
    t.e = 0;
    mt_e = (int)((p.rows + tile_i - 1) / tile_i);
    part = w / (mt_e * ntj);
    t.out_e = part;
    local = w - part * mt_e * ntj;
  }
  if (p.seg != nullptr) {
    // wgrad may have started before its stream's previous kernel ended, so without the wait that makes
    // earlier kernels' writes visible to plain loads: the table, which is complete by then, is read
    // past the L1, which could hold an earlier call's
    seg_row = kMode == kMmWgrad ? 0 : p.seg[2 * t.e];
    seg_rows = kMode == kMmWgrad ? __ldcg(p.seg + 2 * t.e + 1) : p.seg[2 * t.e + 1];
  }
  const int block = local / (kRasterRows * ntj);
  const int in_block = local - block * kRasterRows * ntj;
  const int left_rows = mt_e - block * kRasterRows;
  const int width = left_rows < kRasterRows ? left_rows : kRasterRows;
  const int nt = in_block / width;
  const int mt = block * kRasterRows + in_block - nt * width;
  t.b0 = nt * tile_j;
  if constexpr (kMode == kMmWgrad) {
    t.a0 = mt * tile_i;
    t.out_row = (int64_t)t.e * p.I + t.a0;
    t.rows_valid = p.I - t.a0 < tile_i ? p.I - t.a0 : tile_i;
    t.steps = (int)((seg_rows + kBK - 1) / kBK);
  } else {
    // the segment's rows in equal shares of whole 32 (16 with 16-row tiles): no tile is a small rest
    const int64_t grain = tile_i < 32 ? tile_i : 32;
    const int64_t share = ((seg_rows + mt_e - 1) / mt_e + grain - 1) / grain * grain;
    const int64_t left = seg_rows - mt * share;
    t.a0 = seg_row + (int)(mt * share);
    t.out_row = t.a0;
    t.rows_valid = left < share ? (int)left : (int)share;
    t.steps = (p.R + kBK - 1) / kBK;
  }
  t.k0 = 0;
  if (p.split > 1) {                         // at most 2^19 steps and 74 parts
    t.k0 = t.steps * part / p.split;
    t.steps = t.steps * (part + 1) / p.split - t.k0;
  }
  return t;
}

// Token rows of a tile as the instruction's N: 32, 64, ... 256.
__device__ __forceinline__ int pair_columns(int rows) { return (rows + 31) & ~31; }

constexpr int kPieceBytes = 32 * 128;    // 32 rows of 128 bytes, 128-byte swizzle

// Stores 128 bytes of each of 32 rows (this lane's: w) at column c0, row c1 of matrix c2, through the
// warp's two pieces of shared memory in turn.
__device__ __forceinline__ void store_piece(const void* tmap, uint8_t* pieces, int& turn, const uint32_t* w, int c0,
                                            int c1, int c2, int lane) {
  uint8_t* piece = pieces + turn * kPieceBytes;
  turn ^= 1;
  if (lane == 0) bulk_wait_read1();          // the piece stored from here before has been read
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint4*>(piece + lane * 128 + ((i ^ (lane & 7)) << 4)) =
        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(tmap, piece, c0, c1, c2);
    bulk_commit();
  }
}

// Forward, dgrad: features f0 on of a tile, one per lane of the warp's quarter of the accumulator, the token columns
// first, first + step, ... 32 at a time.
__device__ __forceinline__ void store_tokens(const MmArgs& p, const void* map_y, const void* map_z, uint32_t acc,
                                             const Tile& t, int f0, int first, int step, int most, uint8_t* pieces,
                                             int& turn, int lane) {
  const bool col_ok = f0 + (lane & 3) * 8 < p.J;      // J is a multiple of 8
  float bias[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int f = f0 + 8 * b + (lane >> 2);
    bias[b] = p.bias != nullptr && f < p.J ? __ldg(p.bias + f) : 0.0f;
  }
  // the next piece's accumulator values and residual are on their way while one is stored; one copy of
  // the code for all pieces, since straight-line code for all four ran at the rate of the instruction fetches
  uint32_t v[2][16];
  uint4 res[4];
  auto fetch = [&](int c) {
    if (c >= most || c >= t.rows_valid) return;
    tmem_ld_16x256b_x4(acc + c, v[0]);
    tmem_ld_16x256b_x4(acc + (16u << 16) + c, v[1]);
    if (p.residual != nullptr) {
      const uint16_t* from = static_cast<const uint16_t*>(p.residual) + f0 + (lane & 3) * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = c + i * 8 + (lane >> 2);
        res[i] = col_ok && r < t.rows_valid ? *reinterpret_cast<const uint4*>(from + (t.out_row + r) * (int64_t)p.J)
                                            : make_uint4(0, 0, 0, 0);
      }
    }
  };
  fetch(first);
  with_act(p.act, p.fp16 != 0, [&](auto act, auto fp16) {
#pragma unroll 1
    for (int c = first; c < t.rows_valid; c += step) {
      tmem_ld_wait();
      const PieceAt to{map_y, map_z, t.out_row + c, f0, t.rows_valid - c};
      store_piece32<decltype(act)::value, decltype(fp16)::value>(p, to, pieces, turn, v, bias, res, lane,
                                                                 [&] { fetch(c + step); });
    }
  });
}

// Tiles are handed out from a counter of the grid (the first is the pair's own index): tiles differ
// in cost, so a fixed assignment left pairs idle (64 experts of skewed sizes, 32768 rows: 803 us).
constexpr int kWorkRing = 4;             // tiles the loads may run ahead of the epilogue

struct __align__(1024) PairSmem {
  uint8_t a[kPairStages][kOperandBytes];
  uint8_t b[kPairStages][kOperandBytes];
  // wgrad: two pieces of 4 KB a warp (1024-byte aligned); forward, dgrad: four token pieces
  uint8_t epi[kPairEpiWarps * 2 * kPieceBytes];
  uint64_t full[kPairStages];        // (first CTA) both CTAs' loads of the stage have landed
  uint64_t empty[kPairStages];   // the MMAs have read the stage
  uint64_t acc_full[2];
  uint64_t acc_empty[2];         // (first CTA) both CTAs' epilogues have read the accumulator
  uint64_t drain;
  uint64_t work_full[kWorkRing];     // the slot's tile has arrived
  uint64_t work_empty[kWorkRing];    // (first CTA) every reader in both CTAs has it
  int work[kWorkRing];               // tile index, -1: no more
  uint32_t tmem_base;
  int abort_flag;
};

// The next tile of a reader (a whole warp, or one thread): -1 when there are no more, -2 when the wait
// ran out.  Frees the slot once every lane has read it.
template <bool kWarp>
__device__ __forceinline__ int next_tile(PairSmem& s, int it, int lane, uint64_t limit_ns) {
  const int slot = it & (kWorkRing - 1);
  bool got = wait_cluster(&s.work_full[slot], (uint32_t)(it / kWorkRing) & 1u, &s.abort_flag, limit_ns);
  if (kWarp) got = __all_sync(0xffffffffu, got);
  if (!got) return -2;
  const int w = *reinterpret_cast<volatile int*>(&s.work[slot]);
  if (kWarp) __syncwarp();
  if (!kWarp || lane == 0) mbar_arrive_rank(&s.work_empty[slot], 0);
  return w;
}

template <int kMode>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
mm_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ CUtensorMap map_b64, const __grid_constant__ CUtensorMap map_b32,
               const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_z,
               const __grid_constant__ MmArgs p) {
  // forward, dgrad: A = the weights (i: output features), B = the token rows (j)
  constexpr bool kTokens = kMode != kMmWgrad;
  constexpr bool kAMn = kMode != kMmForward;
  constexpr bool kBMn = kMode == kMmWgrad;
  extern __shared__ uint8_t smem_raw[];
  PairSmem& s = *reinterpret_cast<PairSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();

  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], 2 * kPairEpiWarps);
    }
    mbar_init(&s.drain, 1);
    for (int i = 0; i < kWorkRing; ++i) {
      mbar_init(&s.work_full[i], 1);
      // MMA issuer, the second CTA's loads, both CTAs' epilogue warps
      mbar_init(&s.work_empty[i], 2 + 2 * kPairEpiWarps);
    }
    s.abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&map_a);
    prefetch_tmap(&map_b);
  }
  if (warp == 1) tmem_alloc_pair(&s.tmem_base, 512);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (!p.late_wait) pdl_wait();
  if (p.reset_status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;
  pdl_trigger();

  const uint32_t tmem = s.tmem_base;
  const int tile_i = kTokens ? p.plan.tile_rows : kPairTile;
  const int total = total_tiles<kMode>(p, tile_i, kPairTile);
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------------------------------------- loads ----
    __syncwarp();
    if (elect_one()) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      int next = pair, after = -1, map_e = -1;
      for (int it = 0; ok; ++it) {
        const int slot = it & (kWorkRing - 1);
        int w;
        if (rank == 0) {
          if (!wait_cluster(&s.work_empty[slot], ((uint32_t)(it / kWorkRing) & 1u) ^ 1u, &s.abort_flag, p.wait_ns)) {
            set_abort(&s.abort_flag, p.status);
            ok = false;
            break;
          }
          w = next < total ? next : -1;
          // the ones after it are asked for two tiles ahead, so that the answers are there in time
          if (p.work_counter == nullptr) {
            next += pairs;
          } else if (w >= 0) {
            next = it == 0 ? pairs + atomicAdd(p.work_counter, 1) : after;
            after = pairs + atomicAdd(p.work_counter, 1);
          }
          store_rank(&s.work[slot], &s.work_full[slot], 1, w);
          s.work[slot] = w;
          mbar_arrive(&s.work_full[slot]);
        } else {
          mbar_arrive_expect_tx(&s.work_full[slot], 4);
          w = next_tile<false>(s, it, lane, p.wait_ns);
          if (w == -2) {
            set_abort(&s.abort_flag, p.status);
            ok = false;
          }
        }
        if (w < 0) break;
        if (p.skip_loads == (int)blockIdx.x + 1) {           // test hook: what these loads would bring never comes
          ok = false;
          break;
        }
        const Tile t = tile_at<kMode>(p, w, tile_i, kPairTile);
        // wgrad: 128 rows of each operand; else 128 features, and half of the tile's token rows in
        // the smallest box that covers them
        const int half = kTokens ? pair_columns(t.rows_valid) / 2 : kHalf;
        const int ai = (kTokens ? t.b0 : t.a0) + (int)rank * kHalf;
        const int bj = (kTokens ? t.a0 : t.b0) + (int)rank * half;
        const void* ma = &map_a;
        const void* mb = half > 64 ? &map_b : half > 32 ? &map_b64 : &map_b32;
        if (!kTokens && p.seg_maps != nullptr && t.steps > 0) {
          ma = p.seg_maps + 2 * t.e;
          mb = p.seg_maps + 2 * t.e + 1;
          if (t.e != map_e) {
            acquire_tmap(ma);
            acquire_tmap(mb);
            map_e = t.e;
          }
        }
        const uint32_t b_bytes = (half > 64 ? kHalf : half > 32 ? 64 : 32) * kBK * 2;
        for (int k = 0; k < t.steps; ++k) {
          if (!wait_cluster(&s.empty[stage], phase ^ 1u, &s.abort_flag, p.wait_ns)) {
            set_abort(&s.abort_flag, p.status);
            ok = false;
            break;
          }
          const uint32_t bar = map_rank(smem_u32(&s.full[stage]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&s.full[stage], 2 * (kOperandBytes + b_bytes));
          const int r = (t.k0 + k) * kBK;
          const int ae = kTokens ? t.e : 0;
          if constexpr (kAMn) {
            tma_load_pair(s.a[stage], ma, bar, ai, r, ae);
            tma_load_pair(s.a[stage] + kOperandBytes / 2, ma, bar, ai + 64, r, ae);
          } else {
            tma_load_pair(s.a[stage], ma, bar, r, ai, ae);
          }
          if constexpr (kBMn) {
            tma_load_pair(s.b[stage], mb, bar, bj, r, 0);
            tma_load_pair(s.b[stage] + kOperandBytes / 2, mb, bar, bj + 64, r, 0);
          } else {
            tma_load_pair(s.b[stage], mb, bar, r, bj, 0);
          }
          if (++stage == kPairStages) { stage = 0; phase ^= 1u; }
        }
      }
      // The MMAs' completion arrives on both CTAs' `empty` barriers asynchronously, and nothing else of
      // this CTA waits for the last of those arrivals: without this one could reach the shared memory
      // of a CTA that has exited, or of the next kernel's.  It also shows that every copy has landed.
      for (int i = 0; ok && i < kPairStages; ++i) {
        if (!wait_cluster(&s.empty[stage], phase ^ 1u, &s.abort_flag, p.wait_ns)) {
          set_abort(&s.abort_flag, p.status);
          ok = false;
        }
        if (++stage == kPairStages) { stage = 0; phase ^= 1u; }
      }
      // A pair that gives up does not know what is under way: a millisecond for it to arrive.
      if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(10000);
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMAs ----
    __syncwarp();
    if (rank == 0 && elect_one()) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      int it = 0;                            // tiles with an accumulator
      for (int n = 0; ok; ++n) {
        const int w = next_tile<false>(s, n, lane, p.wait_ns);
        if (w < 0) {
          if (w == -2) set_abort(&s.abort_flag, p.status);
          break;
        }
        const Tile t = tile_at<kMode>(p, w, tile_i, kPairTile);
        if (t.steps == 0) continue;
        const uint32_t idesc =
            idesc_f16(2 * kHalf, kTokens ? pair_columns(t.rows_valid) : kPairTile, p.fp16 != 0, kAMn, kBMn);
        const uint32_t acc = tmem + (uint32_t)(it & 1) * kPairTile;
        if (!wait_cluster(&s.acc_empty[it & 1], ((uint32_t)(it >> 1) & 1u) ^ 1u, &s.abort_flag, p.wait_ns)) {
          set_abort(&s.abort_flag, p.status);
          break;
        }
        tc_fence_after();
        for (int k = 0; k < t.steps; ++k) {
          if (!wait_cluster(&s.full[stage], phase, &s.abort_flag, p.wait_ns)) {
            set_abort(&s.abort_flag, p.status);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(s.a[stage]), b0 = smem_u32(s.b[stage]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // 16 values along r: 32 bytes of a K-major line, 16 lines of an MN-major tile
            const uint64_t da = kAMn ? desc_mn_sw128(a0 + 2048 * j, kOperandBytes / 2) : desc_k_sw128(a0 + 32 * j);
            const uint64_t db = kBMn ? desc_mn_sw128(b0 + 2048 * j, kOperandBytes / 2) : desc_k_sw128(b0 + 32 * j);
            mma_f16_pair(acc, da, db, idesc, (k | j) != 0 ? 1u : 0u);
          }
          tc_commit_pair(&s.empty[stage]);
          if (++stage == kPairStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        tc_commit_pair(&s.acc_full[it & 1]);
        ++it;
      }
      // every tensor-core operation of the pair is done before the memories are given back
      tc_commit_pair_local(&s.drain);
      if (!mbar_wait(&s.drain, 0)) set_abort(&s.abort_flag, p.status);
    }
  } else if (warp >= 4) {
    // ----------------------------------------------------------- epilogue ----
    const int q = warp & 3;                  // tensor-memory lane quarter this warp may read
    const int part = (warp - 4) >> 2;        // which of the quarter's two warps
    uint8_t* pieces = s.epi + (warp - 4) * 2 * kPieceBytes;
    int turn = 0;
    int it = 0;                              // tiles with an accumulator
    for (int n = 0;; ++n) {
      const int w = next_tile<true>(s, n, lane, p.wait_ns);
      if (w < 0) {
        if (w == -2) set_abort(&s.abort_flag, p.status);
        break;
      }
      const Tile t = tile_at<kMode>(p, w, tile_i, kPairTile);
      const bool has_acc = t.steps > 0;
      if (has_acc) {
        const bool got = wait_cluster(&s.acc_full[it & 1], (uint32_t)(it >> 1) & 1u, &s.abort_flag, p.wait_ns);
        if (__any_sync(0xffffffffu, !got)) {
          set_abort(&s.abort_flag, p.status);
          break;
        }
        tc_fence_after();
      }
      const uint32_t acc = tmem + (uint32_t)(it & 1) * kPairTile + ((uint32_t)(q * 32) << 16);
      const int lane0 = (int)rank * kHalf + q * 32;        // this warp's first accumulator lane in the tile
      // the warps of a quarter take its 32-column pieces in turn
      if constexpr (kTokens) {
        if (p.parts != nullptr) {              // sums of a part: FP32, a feature per lane
          const int f = t.b0 + lane0 + lane;
#pragma unroll 1
          for (int c = 32 * part; c < t.rows_valid; c += 64) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(acc + c, v);
            tmem_ld_wait();
            float* to = p.parts + ((int64_t)t.out_e * p.rows + t.out_row + c) * p.J + f;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (f < p.J && c + i < t.rows_valid) to[(int64_t)i * p.J] = __uint_as_float(v[i]);
          }
        } else if (t.b0 + lane0 < p.J) {
          store_tokens(p, &map_out, &map_z, acc, t, t.b0 + lane0, 32 * part, 64, kPairTile, pieces, turn, lane);
        }
      } else {
        // this warp's 64-column pieces, all in registers before any is stored, so that the accumulator is
        // free early
        uint32_t v[2][64];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (has_acc) {
            tmem_ld_32x32b_x32(acc + 64 * part + 128 * j, v[j]);
            tmem_ld_32x32b_x32(acc + 64 * part + 128 * j + 32, v[j] + 32);
          } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) v[j][i] = 0u;
          }
        }
        if (has_acc) {
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_rank(&s.acc_empty[it & 1], 0);
          ++it;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = t.b0 + 64 * part + 128 * j, row = t.a0 + lane0;
          // rows and columns behind the output's are clipped by the map
          if (lane0 >= t.rows_valid || col >= p.J) continue;
          if (p.out_f32) {
            store_piece(&map_out, pieces, turn, v[j], col, row, t.out_e, lane);
            if (col + 32 < p.J) store_piece(&map_out, pieces, turn, v[j] + 32, col + 32, row, t.out_e, lane);
          } else {
            uint32_t h[32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              h[i] = pack16(__uint_as_float(v[j][2 * i]), __uint_as_float(v[j][2 * i + 1]), p.fp16 != 0);
            store_piece(&map_out, pieces, turn, h, col, row, t.out_e, lane);
          }
        }
      }
      if (kTokens && has_acc) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_rank(&s.acc_empty[it & 1], 0);
        ++it;
      }
    }
    if (lane == 0) bulk_wait_all0();
  }

  __syncwarp();
  spread_abort(&s.abort_flag, 2);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
  // the pair gives its tensor memory back together: neither CTA exits before the other has
  __syncwarp();
  cluster_sync();
  if (p.late_wait) pdl_wait();
}

// ------------------------------------------------------------- few rows ----
// Products with few token rows per segment (decode, small experts) read the weights once and little
// else, so the weights are the 128-row operand and the tokens the narrow one: a tile is 128 output
// columns x kTok token rows, D^T[j][i] = sum_r W[j][r] x[i][r], on one CTA (cta_group::1).  16 KB of
// weights arrive per 64-deep step through a deep ring, which keeps enough loads in flight for
// HBM; padding the tokens to kTok costs tensor time only.  When there are fewer tiles than SMs, a
// cluster of `split` CTAs shares a tile's reduction: each adds its part of the steps, the parts meet
// in distributed shared memory and each CTA sums and stores some of the token rows, in rank order
// (a fixed order of additions, no workspace).
constexpr int kNarrowThreads = 256;
constexpr int kMaxSplit = 6;
// Clusters of `split` such CTAs (one an SM) that fit a B200 at once: a cluster stays inside a GPC, so
// fewer than 148 / split.  More would run as a second wave.
__host__ __device__ constexpr int clusters_that_fit(int split) {
  return split == 1 ? 148 : split == 2 ? 74 : split == 3 ? 44 : split == 4 ? 32 : split == 5 ? 25 : 21;
}

template <int kTok>
struct NarrowCfg {
  static constexpr int kStages = kTok <= 16 ? 10 : kTok <= 32 ? 9 : kTok <= 64 ? 7 : 5;
  static constexpr uint32_t kAccCols = kTok < 32 ? 32 : kTok;      // the epilogue reads 32 at a time
  static constexpr uint32_t kTmemCols = 2 * kAccCols;
  static constexpr int kPartRows = kTok < 64 ? 64 : kTok;
};

template <int kTok>
struct __align__(1024) NarrowSmem {
  uint8_t w[NarrowCfg<kTok>::kStages][kOperandBytes];
  uint8_t x[NarrowCfg<kTok>::kStages][kTok * kBK * 2];
  // split > 1: this CTA's sums of the tile, token-major; else four token pieces a warp
  float part[NarrowCfg<kTok>::kPartRows][kHalf];
  uint64_t full[NarrowCfg<kTok>::kStages];
  uint64_t empty[NarrowCfg<kTok>::kStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t part_full;                 // every CTA of the cluster has written its part
  uint64_t part_empty;                // every CTA has read this CTA's part
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ void tma_load_cta(void* dst, const void* tmap, uint64_t* bar, int32_t c0, int32_t c1,
                                             int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ void mma_f16_cta(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <int kMode, int kTok>
__global__ void __launch_bounds__(kNarrowThreads, 1)
mm_narrow_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                 const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_z,
                 const __grid_constant__ MmArgs p, int split) {
  using C = NarrowCfg<kTok>;
  constexpr int kStages = C::kStages;
  constexpr bool kWMn = kMode == kMmDgrad;
  constexpr int kXBytes = kTok * kBK * 2;
  extern __shared__ uint8_t smem_raw[];
  NarrowSmem<kTok>& s = *reinterpret_cast<NarrowSmem<kTok>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                             ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = split > 1 ? (int)cluster_rank() : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], 4);
    }
    mbar_init(&s.part_full, 4 * split);
    mbar_init(&s.part_empty, 4 * split);
    mbar_init(&s.drain, 1);
    s.abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&map_w);
    prefetch_tmap(&map_x);
  }
  if (warp == 1) {
    tmem_alloc(&s.tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  if (split > 1) cluster_sync(); else __syncthreads();
  tc_fence_after();
  if (!p.late_wait) pdl_wait();
  if (p.reset_status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;
  pdl_trigger();

  const uint32_t tmem = s.tmem_base;
  const int total = total_tiles<kMode>(p, kTok, kHalf);
  const int first = blockIdx.x / split, step = gridDim.x / split;
  const int all_steps = (p.R + kBK - 1) / kBK;
  // this CTA's part of every tile's reduction (at least one step: split <= all_steps)
  const int k0 = (int)((int64_t)all_steps * rank / split), k1 = (int)((int64_t)all_steps * (rank + 1) / split);

  if (warp == 0) {
    // ------------------------------------------------------------- loads ----
    __syncwarp();
    if (elect_one()) {
      uint32_t stage = 0, phase = 0, issued = 0, issued_par = 0;
      bool ok = true;
      for (int w = first; ok && w < total; w += step) {
        if (p.skip_loads == (int)blockIdx.x + 1) {           // test hook, as in the pairs
          ok = false;
          break;
        }
        const Tile t = tile_at<kMode>(p, w, kTok, kHalf);
        for (int k = k0; k < k1; ++k) {
          if (!wait_cluster(&s.empty[stage], phase ^ 1u, &s.abort_flag, p.wait_ns)) {
            set_abort(&s.abort_flag, p.status);
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&s.full[stage], kOperandBytes + kXBytes);
          const int r = k * kBK;
          if constexpr (kWMn) {
            tma_load_cta(s.w[stage], &map_w, &s.full[stage], t.b0, r, t.e);
            tma_load_cta(s.w[stage] + kOperandBytes / 2, &map_w, &s.full[stage], t.b0 + 64, r, t.e);
          } else {
            tma_load_cta(s.w[stage], &map_w, &s.full[stage], r, t.b0, t.e);
          }
          tma_load_cta(s.x[stage], &map_x, &s.full[stage], r, t.a0, 0);
          issued |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
      // the MMAs have read every stage: no copy and no arrival of theirs is under way at the exit
      for (int i = 0; ok && i < kStages; ++i) {
        if (!wait_cluster(&s.empty[stage], phase ^ 1u, &s.abort_flag, p.wait_ns)) {
          set_abort(&s.abort_flag, p.status);
          ok = false;
        }
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
      // after giving up, the copies at least have landed
      for (int i = 0; !ok && i < kStages; ++i)
        if ((issued >> i) & 1u)
          if (!mbar_wait(&s.full[i], (issued_par >> i) & 1u)) set_abort(&s.abort_flag, p.status);
    }
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMAs ----
    __syncwarp();
    if (elect_one()) {
      uint32_t stage = 0, phase = 0;
      const uint32_t idesc = idesc_f16(kHalf, kTok, p.fp16 != 0, kWMn, false);
      bool ok = true;
      int it = 0;
      for (int w = first; ok && w < total; w += step, ++it) {
        const uint32_t acc = tmem + (uint32_t)(it & 1) * C::kAccCols;
        if (!wait_cluster(&s.acc_empty[it & 1], ((uint32_t)(it >> 1) & 1u) ^ 1u, &s.abort_flag, p.wait_ns)) {
          set_abort(&s.abort_flag, p.status);
          break;
        }
        tc_fence_after();
        for (int k = k0; k < k1; ++k) {
          if (!wait_cluster(&s.full[stage], phase, &s.abort_flag, p.wait_ns)) {
            set_abort(&s.abort_flag, p.status);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t w0 = smem_u32(s.w[stage]), x0 = smem_u32(s.x[stage]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t dw = kWMn ? desc_mn_sw128(w0 + 2048 * j, kOperandBytes / 2) : desc_k_sw128(w0 + 32 * j);
            mma_f16_cta(acc, dw, desc_k_sw128(x0 + 32 * j), idesc, k != k0 || j != 0 ? 1u : 0u);
          }
          tc_commit(&s.empty[stage]);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        tc_commit(&s.acc_full[it & 1]);
      }
      // every tensor-core operation is done before the memories are given back
      tc_commit(&s.drain);
      if (!mbar_wait(&s.drain, 0)) set_abort(&s.abort_flag, p.status);
    }
  } else if (warp >= 4) {
    // ----------------------------------------------------------- epilogue ----
    const int q = warp & 3;
    static_assert(sizeof(s.part) >= 16 * kTokenPiece, "the epilogue's pieces");
    uint8_t* pieces = reinterpret_cast<uint8_t*>(s.part) + q * 4 * kTokenPiece;
    int it = 0, turn = 0;
    for (int w = first; w < total; w += step, ++it) {
      const Tile t = tile_at<kMode>(p, w, kTok, kHalf);
      if (split == 1) {                      // each warp by itself
        const bool got = wait_cluster(&s.acc_full[it & 1], (uint32_t)(it >> 1) & 1u, &s.abort_flag, p.wait_ns);
        if (__any_sync(0xffffffffu, !got)) {
          set_abort(&s.abort_flag, p.status);
          break;
        }
        tc_fence_after();
        if (t.b0 + q * 32 < p.J)
          store_tokens(p, &map_out, &map_z, tmem + (uint32_t)(it & 1) * C::kAccCols + ((uint32_t)(q * 32) << 16), t,
                       t.b0 + q * 32, 0, 32, kTok, pieces, turn, lane);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.acc_empty[it & 1]);
        continue;
      }
      bool got = wait_cluster(&s.acc_full[it & 1], (uint32_t)(it >> 1) & 1u, &s.abort_flag, p.wait_ns);
      // the tile before this one has been read by every CTA of the cluster
      if (it > 0) got = got && wait_cluster(&s.part_empty, (uint32_t)(it - 1) & 1u, &s.abort_flag, p.wait_ns);
      if (__any_sync(0xffffffffu, !got)) {
        set_abort(&s.abort_flag, p.status);
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(it & 1) * C::kAccCols + ((uint32_t)(q * 32) << 16);
#pragma unroll
      for (int c = 0; c < kTok; c += 16) {
        if (c >= t.rows_valid) break;
        uint32_t v[16];
        tmem_ld_32x32b_x16(acc + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) s.part[c + i][q * 32 + lane] = __uint_as_float(v[i]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.acc_empty[it & 1]);
      if (lane < split) mbar_arrive_rank_release(&s.part_full, lane);
      const bool all = wait_cluster(&s.part_full, (uint32_t)it & 1u, &s.abort_flag, p.wait_ns);
      if (__any_sync(0xffffffffu, !all)) {
        set_abort(&s.abort_flag, p.status);
        break;
      }
      const int col = t.b0 + 4 * lane;
      if (col < p.J) {                     // J is a multiple of 8
        const float4 bias = p.bias != nullptr ? __ldg(reinterpret_cast<const float4*>(p.bias + col))
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
        const int64_t at0 = t.out_row * (int64_t)p.J + col;
        with_act(p.act, p.fp16 != 0, [&](auto act, auto fp16) {
          // four rows at a time: their residual loads and the reads of the parts overlap
          for (int r0 = rank + split * q; r0 < t.rows_valid; r0 += 16 * split) {
            uint2 res[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = r0 + 4 * split * i;
              res[i] = p.residual != nullptr && r < t.rows_valid
                           ? *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.residual) + at0 +
                                                             r * (int64_t)p.J)
                           : make_uint2(0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = r0 + 4 * split * i;
              if (r >= t.rows_valid) continue;
              float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
              const uint32_t at = smem_u32(&s.part[r][4 * lane]);
              for (int c = 0; c < split; ++c) {
                const float4 o = ld_cluster_f4(map_rank(at, c));
                v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
              }
              store4<decltype(act)::value, decltype(fp16)::value>(p, v, bias, res[i], at0 + r * (int64_t)p.J);
            }
          }
        });
      }
      __syncwarp();
      if (lane < split) mbar_arrive_rank(&s.part_empty, lane);
    }
    if (lane == 0) bulk_wait_all0();
  }

  __syncwarp();
  spread_abort(&s.abort_flag, split);
  tc_fence_before();
  if (split > 1) cluster_sync(); else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
  if (p.late_wait) pdl_wait();
}

// One thread per expert: its segment from the offsets, and the scan of the row tiles; then, for wgrad,
// one warp per tensor map: a one-row map of the operand with the segment's first row and row count.
__global__ void __launch_bounds__(kMaxGroups) mm_table_kernel(const int32_t* offsets, int E, int64_t rows,
                                                              int tile_rows, MmTable t, WsHeader* hdr,
                                                              const __grid_constant__ MmSegMaps maps) {
  __shared__ int warp_sum[32];
  __shared__ __align__(128) uint32_t s_map[32][32];
  pdl_wait();
  pdl_trigger();
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  int64_t lo = 0, hi = 0;
  if (offsets != nullptr && e < E) {
    lo = offsets[e];
    hi = offsets[e + 1];
  }
  const bool bad = __syncthreads_or(lo < 0 || hi < lo || hi > rows);
  if (e == 0) {
    hdr->status = bad ? kStatusBadInput : 0u;
    hdr->work[0] = hdr->work[1] = 0;
  }
  if (offsets == nullptr) return;
  if (bad) lo = hi = 0;
  const int n = (int)((hi - lo + tile_rows - 1) / tile_rows);
  int sum = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += up;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < warp; ++i) before += warp_sum[i];
  if (e < E) {
    t.seg[2 * e] = (int)lo;
    t.seg[2 * e + 1] = (int)(hi - lo);
    t.tiles[e + 1] = before + sum;
  }
  if (e == 0) t.tiles[0] = 0;
  if (maps.out == nullptr) return;
  __syncthreads();                        // the segments are written (read back below)
  for (int m = warp; m < 2 * E; m += blockDim.x >> 5) {
    const int which = m & 1;
    // an empty segment's map is never loaded from; it is a valid one all the same
    const int rows_of = t.seg[2 * (m >> 1) + 1], count = rows_of > 0 ? rows_of : 1;
    const int first = rows_of > 0 ? t.seg[2 * (m >> 1)] : 0;
    __syncwarp();
    s_map[warp][lane] = reinterpret_cast<const uint32_t*>(which == 0 ? &maps.a : &maps.b)[lane];
    __syncwarp();
    const uint32_t at = smem_u32(s_map[warp]);
    if (lane == 0) {
      const uint64_t base = reinterpret_cast<uint64_t>(which == 0 ? maps.a_base : maps.b_base) +
                            (uint64_t)first * (uint64_t)(which == 0 ? maps.a_row_bytes : maps.b_row_bytes);
      asm volatile("tensormap.replace.tile.global_address.shared::cta.b1024.b64 [%0], %1;" ::"r"(at), "l"(base)
                   : "memory");
      asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(at), "r"(count)
                   : "memory");
    }
    __syncwarp();
    asm volatile(
        "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
            maps.out + m),
        "r"(at)
        : "memory");
  }
}

template <int kMode>
cudaError_t launch_pair(const void* a, const void* b, const MmArgs& args, cudaStream_t stream) {
  MmArgs m = args;
  if (m.split <= 1) {
    m.split = 1;
    m.parts = nullptr;
  } else if (m.parts == nullptr || (kMode != kMmWgrad && m.seg != nullptr)) {
    return cudaErrorInvalidValue;
  }
  if (kMode == kMmWgrad && m.split > 1) {
    m.out = m.parts;
    m.out_f32 = 1;
  }
  const int tile_rows = m.plan.tile_rows;
  CUtensorMap map_a, map_b, map_b64, map_b32, map_out, map_z;
  int err;
  if (kMode == kMmWgrad) {
    err = make_tma_16(&map_a, a, m.I, m.rows, 1, kBK) | make_tma_16(&map_b, b, m.J, m.rows, 1, kBK) |
          make_tma_3d(&map_out, m.out, m.out_f32 ? 4 : 2, m.J, m.I, (uint64_t)m.split * m.E, 32, 128);
    map_b64 = map_b32 = map_z = map_b;                 // not used
  } else {
    err = kMode == kMmForward ? make_tma_16(&map_a, b, m.R, m.J, m.E, kHalf)
                              : make_tma_16(&map_a, b, m.J, m.R, m.E, kBK);
    err |= make_tma_16(&map_b, a, m.R, m.rows, 1, kHalf) | make_tma_16(&map_b64, a, m.R, m.rows, 1, 64) |
           make_tma_16(&map_b32, a, m.R, m.rows, 1, 32);
    err |= make_tma_3d(&map_out, m.out, 2, m.J, m.rows, 1, 32, 64);
    map_z = map_out;
    if (m.z_out != nullptr) err |= make_tma_3d(&map_z, m.z_out, 2, m.J, m.rows, 1, 32, 64);
  }
  if (err != 0) return cudaErrorInvalidValue;
  const size_t smem = sizeof(PairSmem) + 1024;
  static_assert(sizeof(PairSmem) + 1024 <= 232448, "shared memory exceeds the per-block limit");
  static_assert(4 * kTokenPiece <= 2 * kPieceBytes, "the epilogue's pieces");
  const cudaError_t ce = allow_smem(reinterpret_cast<const void*>(mm_pair_kernel<kMode>), smem);
  if (ce != cudaSuccess) return ce;
  const int64_t ntj = (m.J + kPairTile - 1) / kPairTile;
  int64_t most = kMode == kMmWgrad ? (int64_t)m.E * ((m.I + kPairTile - 1) / kPairTile)
                                   : (m.rows + tile_rows - 1) / tile_rows + (m.seg != nullptr ? m.E : 0);
  most *= ntj * m.split;
  const int64_t pairs = num_sms() / 2;
  return launch_pdl(mm_pair_kernel<kMode>, dim3((unsigned)(2 * (most < pairs ? most : pairs))), dim3(kPairThreads),
                    smem, stream, map_a, map_b, map_b64, map_b32, map_out, map_z, m);
}

template <int kMode, int kTok>
cudaError_t launch_narrow(const void* a, const void* b, const MmArgs& m, int split, cudaStream_t stream) {
  CUtensorMap map_w, map_x;
  int err = (kMode == kMmForward ? make_tma_16(&map_w, b, m.R, m.J, m.E, kHalf)
                                 : make_tma_16(&map_w, b, m.J, m.R, m.E, kBK)) |
            make_tma_16(&map_x, a, m.R, m.rows, 1, kTok);
  CUtensorMap map_out = map_x, map_z = map_x;          // used for whole pieces of tiles that are not shared
  if (split == 1 && kTok >= 32) {
    err |= make_tma_3d(&map_out, m.out, 2, m.J, m.rows, 1, 32, 64);
    if (m.z_out != nullptr) err |= make_tma_3d(&map_z, m.z_out, 2, m.J, m.rows, 1, 32, 64);
  }
  if (err != 0) return cudaErrorInvalidValue;
  const size_t smem = sizeof(NarrowSmem<kTok>) + 1024;
  static_assert(sizeof(NarrowSmem<kTok>) + 1024 <= 232448, "shared memory exceeds the per-block limit");
  auto kernel = mm_narrow_kernel<kMode, kTok>;
  const cudaError_t ce = allow_smem(reinterpret_cast<const void*>(kernel), smem);
  if (ce != cudaSuccess) return ce;
  int64_t most = (m.rows + kTok - 1) / kTok;
  if (m.seg != nullptr) most += m.E < m.rows ? m.E : m.rows;
  most *= (m.J + kHalf - 1) / kHalf;
  const int64_t room = clusters_that_fit(split);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((most < room ? most : room) * split));
  cfg.blockDim = dim3(kNarrowThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, map_w, map_x, map_out, map_z, m, split);
}

template <int kMode>
cudaError_t launch_rows(const void* a, const void* b, const MmArgs& m, cudaStream_t stream) {
  if (m.plan.pair) return launch_pair<kMode>(a, b, m, stream);
  switch (m.plan.tile_rows) {
    case 16: return launch_narrow<kMode, 16>(a, b, m, m.plan.split, stream);
    case 32: return launch_narrow<kMode, 32>(a, b, m, m.plan.split, stream);
    case 64: return launch_narrow<kMode, 64>(a, b, m, m.plan.split, stream);
    default: return launch_narrow<kMode, 128>(a, b, m, m.plan.split, stream);
  }
}

// Four neighbouring values a lane, one eighth of their parts a warp: each warp's sum in the parts' order, the
// warps' sums in theirs (an order that the shape fixes), then the product's epilogue.  At most 74 tiles'
// parts, which are in L2: its time is its latency, which one thread per value makes long.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(32 * kJoinWarps) mm_join_kernel(const __grid_constant__ MmArgs p, int n4) {
  __shared__ float4 sums[kJoinWarps][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int at = blockIdx.x * 32 + lane;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (at < n4) {
    const float4* from = reinterpret_cast<const float4*>(p.parts) + at;
    const int last = p.split * (warp + 1) / kJoinWarps;
#pragma unroll 4
    for (int i = p.split * warp / kJoinWarps; i < last; ++i) {
      const float4 o = __ldcg(from + (int64_t)i * n4);
      v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
    }
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || at >= n4) return;
  for (int i = 1; i < kJoinWarps; ++i) {
    const float4 o = sums[i][lane];
    v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
  }
  if (p.out_f32) {
    static_cast<float4*>(p.out)[at] = v;
    return;
  }
  const int col = at % (p.J / 4) * 4;
  uint2 res = make_uint2(0, 0);
  if (p.residual != nullptr) res = static_cast<const uint2*>(p.residual)[at];
  const float4 bias = p.bias != nullptr ? __ldg(reinterpret_cast<const float4*>(p.bias + col))
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
  with_act(p.act, p.fp16 != 0, [&](auto act, auto fp16) {
    store4<decltype(act)::value, decltype(fp16)::value>(p, v, bias, res, (int64_t)at * 4);
  });
}

// Where pairs share reductions: at most this many tiles of parts, one for each pair.
constexpr int kPairs = 74;
// SM clocks of the launch that joins `split` parts of n values, and of writing them.
double join_cost(int split, double n) { return 5000.0 + split * n * 8.0 / 2000.0; }

}  // namespace

// The cheapest of the shapes by a model in SM clocks.  A tile's step takes the time to bring its
// operands in: about 45 bytes a clock and SM, 72 on single CTAs whose weights other row tiles read too (from
// L2; 48 where rows are not whole lines), but then 360 clocks at least.  Waves of tiles follow one another, each as long as its steps or
// the epilogue of the one before; the weights from HBM (3500 bytes a clock) run beside all that.  Measured, us,
// single CTAs (the best of them) and pairs: K = N = 5120: 16 rows 11.3 (split 3 ways) and 19.7, 256 rows 20.7 and
// 22.7, 768 rows 39 and 34; K = N = 2560: 512 rows 13.3 and 14.4; K = 64, 8192 x 8192: 69 and 44; 16 experts of
// 192 rows, K = 5120, N = 2560: 118 and 99.  Over 30 shapes the choice was 2 % slower than the best one.
MmPlan mm_plan(int64_t rows, int E, int J, int R, bool ragged) {
  const int64_t steps = (R + kBK - 1) / kBK;
  // how the rows spread over the experts is known on the device only: evenly, for the model
  const int64_t busy = ragged ? (E < rows ? E : rows) : 1;
  const int64_t mean = busy > 0 ? (rows + busy - 1) / busy : 0;
  MmPlan best{false, 16, 1};
  if (mean == 0) return best;
  const double hbm = (double)busy * J * R * 2.0 / 3500.0;
  const bool whole_lines = R % 64 == 0 && J % 64 == 0;       // the copies' 128-byte rows are lines of the L2
  double best_cost = 1e30;
  auto consider = [&](bool pair, int tile, int split) {
    const int64_t per_seg = (mean + tile - 1) / tile, cols = pair ? kPairTile : kHalf;
    const int64_t tiles = busy * per_seg * ((J + cols - 1) / cols);
    if (pair && split > 1 && tiles * split > kPairs) return;
    const int64_t room = pair ? kPairs : clusters_that_fit(split);
    const int64_t waves = pair && split > 1 ? 1 : (tiles + room - 1) / room;
    const double n = pair ? (double)(((mean + per_seg - 1) / per_seg + 31) / 32 * 32) : (double)tile;
    const bool from_l2 = !pair && split == 1 && per_seg > 1;   // mostly, the weights that another row tile reads too
    double step = (16384.0 + (pair ? 64.0 : 128.0) * n) / (!from_l2 ? 45.0 : whole_lines ? 72.0 : 48.0);
    if (from_l2 && step < 360.0) step = 360.0;
    const double mma = (double)((steps + split - 1) / split) * step;
    const double epilogue = pair ? 2300.0 + 14.0 * n : split == 1 ? 2000.0 + 20.0 * n : 2500.0 + 76.0 * n;
    double cost = mma + (double)(waves - 1) * (mma > epilogue ? mma : epilogue);
    cost = cost < hbm ? hbm + 0.2 * cost : cost + 0.2 * hbm;   // the two overlap, but not wholly
    cost += pair         ? 6000.0 + 6.0 * n + (split > 1 ? join_cost(split, (double)rows * J) : 0.0)
            : split == 1 ? 2500.0 + 5.0 * n
                         : 2500.0 + 25.0 * n + (600.0 + 8.0 * n) * (double)waves;
    if (cost < best_cost) {
      best_cost = cost;
      best = MmPlan{pair, tile, split};
    }
  };
  for (int tile = 16; tile <= 128; tile *= 2) {
    if (tile >= 32 && mean <= tile / 2) break;               // all padding
    for (int split = 1; split <= kMaxSplit && split * 4 <= (steps > 4 ? steps : 4); ++split) consider(false, tile, split);
  }
  for (int tile = kPairTile; tile >= 64; tile -= 32) consider(true, tile, 1);
  // (mean <= 2^25 rows: past 74 tiles nothing is shared)
  if (!ragged && mean <= kPairs * kPairTile)
    for (int tile = kPairTile; tile >= 64; tile -= 32) {
      const int64_t tiles = (mean + tile - 1) / tile * ((J + kPairTile - 1) / kPairTile);
      // the most parts that fit, and half as many
      for (int64_t split = kPairs / tiles < steps / 4 ? kPairs / tiles : steps / 4, i = 0; i < 2 && split > 1;
           ++i, split /= 2)
        consider(true, tile, (int)split);
    }
  return best;
}

// The rows' steps of a tile of wgrad run on one pair, in 2 * 256 clocks each at best (728 with the operands
// brought in); parts of them on the pairs that would have no tile, when that saves more than the join costs.
int mm_wgrad_split(int64_t rows, int E, int I, int J) {
  const int64_t tiles = (int64_t)E * ((I + kPairTile - 1) / kPairTile) * ((J + kPairTile - 1) / kPairTile);
  const int64_t steps = (rows + (int64_t)E * kBK - 1) / ((int64_t)E * kBK);   // of a segment, on average
  int best = 1;
  double best_cost = 728.0 * (double)steps;
  for (int64_t split = kPairs / tiles < steps / 4 ? kPairs / tiles : steps / 4, i = 0; i < 2 && split > 1;
       ++i, split /= 2) {
    const double cost =
        728.0 * (double)((steps + split - 1) / split) + join_cost((int)split, (double)E * (double)I * (double)J);
    if (cost < best_cost) {
      best_cost = cost;
      best = (int)split;
    }
  }
  return best;
}

// At most kPairs / tiles and steps / 4 parts, as the plans; tiles x parts are at most kPairs, so the parts never hold
// more than that many tiles.
size_t mm_row_part_floats(int64_t rows, int J, int R) {
  const int64_t across = ((int64_t)J + kPairTile - 1) / kPairTile, steps = ((int64_t)R + kBK - 1) / kBK;
  const int64_t most = kPairs / across < steps / 4 ? kPairs / across : steps / 4;
  if (most < 2) return 0;
  const int64_t all = (int64_t)kPairs * kPairTile * kPairTile, by_rows = most * rows * (int64_t)J;
  return (size_t)(by_rows < all ? by_rows : all);
}

size_t mm_wgrad_part_floats(int64_t rows, int E, int I, int J) {
  const int64_t tiles = (int64_t)E * ((I + kPairTile - 1) / kPairTile) * ((J + kPairTile - 1) / kPairTile);
  const int64_t steps = (rows + (int64_t)E * kBK - 1) / ((int64_t)E * kBK);
  const int64_t most = kPairs / tiles < steps / 4 ? kPairs / tiles : steps / 4;
  return most < 2 ? 0 : (size_t)(most * E * I * (int64_t)J);
}

cudaError_t launch_mm_table(const int32_t* offsets, int E, int64_t rows, int tile_rows, const MmTable& t,
                            WsHeader* hdr, const MmWgradOperands* w, cudaStream_t stream) {
  MmSegMaps maps{};
  if (w != nullptr) {
    // Encoded for one row, the fewest a loaded segment has, and given the segment's rows on the device.  Through a map
    // that the driver encoded for 128 KB or more, a copy reads memory for elements out of bounds too, from the first
    // 128 KB behind the map's address, which lie inside so large a tensor; through a smaller one it does not.  (Boxes
    // of 64 rows of 992 bytes with one in bounds: 1.2 KB read a box through maps of up to 132 rows, 16.3 KB
    // of 133, 131936 bytes; 0.5 KB where such maps share their address.)  Cut down from a map of the whole operand, a
    // short segment's near the operand's end read up to 128 KB behind it: an illegal address where nothing is mapped.
    if (make_tma_16(&maps.a, w->a, w->I, 1, 1, kBK) != 0 || make_tma_16(&maps.b, w->b, w->J, 1, 1, kBK) != 0)
      return cudaErrorInvalidValue;
    maps.a_base = w->a;
    maps.b_base = w->b;
    maps.a_row_bytes = (int64_t)w->I * 2;
    maps.b_row_bytes = (int64_t)w->J * 2;
    maps.out = t.maps;
  }
  const int threads = offsets == nullptr ? 32 : w != nullptr ? kMaxGroups : (E + 31) / 32 * 32;
  return launch_pdl(mm_table_kernel, dim3(1), dim3(threads), 0, stream, offsets, E, rows, tile_rows, t, hdr, maps);
}

cudaError_t launch_mm(int mode, const void* a, const void* b, const MmArgs& m, cudaStream_t stream) {
  switch (mode) {
    case kMmForward: return launch_rows<kMmForward>(a, b, m, stream);
    case kMmDgrad: return launch_rows<kMmDgrad>(a, b, m, stream);
    default: return launch_pair<kMmWgrad>(a, b, m, stream);
  }
}

cudaError_t launch_mm_join(int mode, const MmArgs& m, cudaStream_t stream) {
  const int64_t n4 = (mode == kMmWgrad ? (int64_t)m.E * m.I : m.rows) * m.J / 4;
  return launch_pdl(mm_join_kernel, dim3((unsigned)((n4 + 31) / 32)), dim3(32 * kJoinWarps), 0, stream, m, (int)n4);
}

}  // namespace nvfp4moe
