// Epilogue of the 16-bit products: accumulator values from registers to global memory, with the
// bias, the stored pre-activation, the activation, the residual and the one rounding.
#pragma once

#include "activation.cuh"
#include "common.cuh"
#include "dense.h"

namespace nvfp4moe {

// Four consecutive output columns of one row; res: the residual's, already loaded (with p.residual).
template <int kAct, bool fp16>
__device__ __forceinline__ void store4(const MmArgs& p, float4 f, float4 bias, uint2 res, int64_t at) {
  float v[4] = {f.x + bias.x, f.y + bias.y, f.z + bias.z, f.w + bias.w};
  if (p.z_out != nullptr)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.z_out) + at) =
        make_uint2(pack16(v[0], v[1], fp16), pack16(v[2], v[3], fp16));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = act_value<kAct>(v[i]);
  if (p.residual != nullptr) {
    const float2 f0 = unpack16(res.x, fp16), f1 = unpack16(res.y, fp16);
    v[0] += f0.x; v[1] += f0.y; v[2] += f1.x; v[3] += f1.y;
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
      make_uint2(pack16(v[0], v[1], fp16), pack16(v[2], v[3], fp16));
}

// ---- 32 features x 32 token rows of one warp, transposed in 16 bits through shared memory ----
// The accumulator holds features along tensor-memory lanes and tokens along columns.  tcgen05.ld
// 16x256b hands it out as 8 x 8 fragments (this thread: feature lane / 4, tokens 2 (lane % 4) and the
// next), which stmatrix.trans stores as token rows of 8 features: 4 shared-memory instructions for the whole
// piece (32 when each thread stores its values one by one).  A token row is 64 bytes in the 64-byte
// swizzle of a TMA store, which takes the piece from there; the swizzle also puts a fragment's 8 rows
// in different banks.  (Against plain 16-byte stores: 4096 x 20480, K = 5120, 592 -> 586 us.)
constexpr int kTokenPiece = 32 * 64;

// Byte of 16-byte chunk c of token row r.
__device__ __forceinline__ uint32_t token_chunk(int r, int c) { return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)); }

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Until all but this thread's last bulk store have read shared memory / all have been written.
__device__ __forceinline__ void bulk_wait_read1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all0() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void tma_store_3d(const void* tmap, const void* src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(tmap),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// 16 lanes x 32 columns: for k = 0..3, lane (i / 4) columns 8k + 2 (i % 4) + {0, 1} in r[4k], r[4k + 1] and
// lane (i / 4 + 8) at the same columns in r[4k + 2], r[4k + 3].
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Features 8 b .. 8 b + 7 of 32 tokens between this warp's piece and fragments (w[k]: tokens 8k .. 8k + 7).
__device__ __forceinline__ void put_fragments(uint32_t piece, int b, const uint32_t* w, int lane) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                   piece + token_chunk(lane, b)),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}
__device__ __forceinline__ void get_fragments(uint32_t piece, int b, uint32_t* w, int lane) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(piece + token_chunk(lane, b))
               : "memory");
}

// The first `live` token rows of a piece to rows of the tensor, 16 bytes a lane.
__device__ __forceinline__ void rows_to_global(uint16_t* base, const uint8_t* piece, int64_t at, int64_t J, int live,
                                               int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    if (r < live)
      *reinterpret_cast<uint4*>(base + at + r * J) = *reinterpret_cast<const uint4*>(piece + token_chunk(r, lane & 3));
  }
}

// Where a piece goes: token row `row` on, feature f0 on (of J); `live` of its rows belong to the tile.
struct PieceAt {
  const void *map_y, *map_z;
  int64_t row;
  int f0;
  int live;
};

// v: the accumulator's 32 x 32 values as two tmem_ld_16x256b_x4 give them; bias[b]: of feature 8 b + lane / 4;
// res: this lane's residual vectors (rows lane / 4, + 8, + 16, + 24, features 8 (lane % 4) on).  pieces: the
// warp's [2][y, z] pieces, used in turn.  next(): called once v and res have been used.
template <int kAct, bool fp16, typename Next>
__device__ __forceinline__ void store_piece32(const MmArgs& p, const PieceAt& to, uint8_t* pieces, int& turn,
                                              const uint32_t (*v)[16], const float* bias, const uint4* res, int lane,
                                              Next next) {
  uint8_t* p_y = pieces + turn * 2 * kTokenPiece;
  uint8_t* p_z = p_y + kTokenPiece;
  turn ^= 1;
  if (lane == 0) bulk_wait_read1();              // what was stored from here before has been read
  __syncwarp();
  if (p.residual != nullptr) {                   // through y's piece: a fragment is read before its place is written
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4*>(p_y + token_chunk(i * 8 + (lane >> 2), lane & 3)) = res[i];
    __syncwarp();
  }
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    float f[8];                                  // tokens 8k + 2 (lane % 4) + {0, 1}, k = 0..3
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(v[b >> 1][4 * k + 2 * (b & 1)]) + bias[b];
      f[2 * k + 1] = __uint_as_float(v[b >> 1][4 * k + 2 * (b & 1) + 1]) + bias[b];
    }
    uint32_t w[4];
    if (p.z_out != nullptr) {
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = pack16(f[2 * k], f[2 * k + 1], fp16);
      put_fragments(smem_u32(p_z), b, w, lane);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = act_value<kAct>(f[i]);
    if (p.residual != nullptr) {
      get_fragments(smem_u32(p_y), b, w, lane);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 r = unpack16(w[k], fp16);
        f[2 * k] += r.x;
        f[2 * k + 1] += r.y;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = pack16(f[2 * k], f[2 * k + 1], fp16);
    put_fragments(smem_u32(p_y), b, w, lane);
  }
  next();
  if (to.live >= 32) {                           // whole pieces: the map clips features behind J
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      if (p.z_out != nullptr) tma_store_3d(to.map_z, p_z, to.f0, (int)to.row, 0);
      tma_store_3d(to.map_y, p_y, to.f0, (int)to.row, 0);
    }
  } else {                                       // a segment's last rows: the rows behind are not this tile's
    __syncwarp();
    if (to.f0 + (lane & 3) * 8 < p.J) {          // J is a multiple of 8
      const int64_t at = to.row * p.J + to.f0 + (lane & 3) * 8;
      if (p.z_out != nullptr) rows_to_global(static_cast<uint16_t*>(p.z_out), p_z, at, p.J, to.live, lane);
      rows_to_global(static_cast<uint16_t*>(p.out), p_y, at, p.J, to.live, lane);
    }
  }
  // One group a piece, an empty one for rows stored by the lanes: the wait above leaves the newest group
  // pending, which then is never that of the piece about to be written.
  if (lane == 0) bulk_commit();
}

}  // namespace nvfp4moe
