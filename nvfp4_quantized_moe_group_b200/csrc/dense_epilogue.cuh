// Epilogue of the 16-bit products: accumulator values from registers to global memory, with the
// bias, the stored pre-activation, the activation, the residual and the one rounding.
#pragma once

#include "activation.cuh"
#include "common.cuh"
#include "dense.h"

namespace nvfp4moe {

// Four consecutive output columns of one row; res: the residual's, already loaded (with p.residual).
template <int kAct>
__device__ __forceinline__ void store4(const MmArgs& p, float4 f, float4 bias, uint2 res, int64_t at) {
  const bool fp16 = p.fp16 != 0;
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
// piece (32 when each thread stores its values one by one).  A token row is 64 bytes, 80 apart: the 8
// rows of a fragment, and 8 lanes' 16-byte reads, fall in different banks.
constexpr int kPieceRow = 80;
constexpr int kTokenPiece = 32 * kPieceRow;

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
                   piece + lane * kPieceRow + b * 16),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}
__device__ __forceinline__ void get_fragments(uint32_t piece, int b, uint32_t* w, int lane) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(piece + lane * kPieceRow + b * 16)
               : "memory");
}

// A piece's token rows (`live` of them, 64 bytes each) between shared memory and rows of the tensor: this
// lane's 16 bytes of rows lane / 4, + 8, + 16, + 24.
__device__ __forceinline__ void rows_to_global(uint16_t* base, const uint8_t* piece, int64_t at, int64_t J, int live,
                                               int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    if (r < live)
      *reinterpret_cast<uint4*>(base + at + r * J) =
          *reinterpret_cast<const uint4*>(piece + r * kPieceRow + (lane & 3) * 16);
  }
}

// v: the accumulator's 32 x 32 values as two tmem_ld_16x256b_x4 give them; bias[b]: of feature 8 b + lane / 4;
// res: this lane's residual vectors (rows as in rows_to_global).  at: first token row, column of this lane's
// 8 features; col_ok: that column lies in the output.
template <int kAct>
__device__ __forceinline__ void store_piece32(const MmArgs& p, uint8_t* pieces, const uint32_t (*v)[16],
                                              const float* bias, const uint4* res, int64_t at, int live, bool col_ok,
                                              int lane) {
  const bool fp16 = p.fp16 != 0;
  uint8_t* p_y = pieces;
  uint8_t* p_z = pieces + kTokenPiece;
  uint8_t* p_r = pieces + 2 * kTokenPiece;
  __syncwarp();                                  // the pieces before have been read
  if (p.residual != nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4*>(p_r + (i * 8 + (lane >> 2)) * kPieceRow + (lane & 3) * 16) = res[i];
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
      get_fragments(smem_u32(p_r), b, w, lane);
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
  __syncwarp();
  if (col_ok) {
    if (p.z_out != nullptr) rows_to_global(static_cast<uint16_t*>(p.z_out), p_z, at, p.J, live, lane);
    rows_to_global(static_cast<uint16_t*>(p.out), p_y, at, p.J, live, lane);
  }
}

}  // namespace nvfp4moe
