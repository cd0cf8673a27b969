// Epilogue of the 16-bit products: accumulator rows from registers to global memory, with the
// bias, the stored pre-activation, the activation, the residual and the one rounding.
#pragma once

#include "activation.cuh"
#include "common.cuh"
#include "dense.h"

namespace nvfp4moe {

// One warp's 32 x 32 FP32 transpose tile; rows 144 bytes apart, so 16-byte reads of 8 lanes in two
// rows fall in different banks.
struct EpilogueTile {
  float v[32][36];
};

// Eight consecutive output columns of one row (16-bit output): at = row * J + col.
__device__ __forceinline__ void store8(const MmArgs& p, float* v, const float* bias8, int64_t at) {
  const bool fp16 = p.fp16 != 0;
  if (p.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += bias8[i];
  }
  if (p.z_out != nullptr)
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.z_out) + at) = make_uint4(
        pack16(v[0], v[1], fp16), pack16(v[2], v[3], fp16), pack16(v[4], v[5], fp16), pack16(v[6], v[7], fp16));
  if (p.act != NVFP4MOE_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_value(v[i], p.act);
  }
  if (p.residual != nullptr) {
    const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.residual) + at);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack16(w[i], fp16);
      v[2 * i] += f.x;
      v[2 * i + 1] += f.y;
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at) = make_uint4(
      pack16(v[0], v[1], fp16), pack16(v[2], v[3], fp16), pack16(v[4], v[5], fp16), pack16(v[6], v[7], fp16));
}

// Four consecutive output columns of one row (16-bit output).
__device__ __forceinline__ void store4(const MmArgs& p, float4 f, int64_t at, int col) {
  const bool fp16 = p.fp16 != 0;
  float v[4] = {f.x, f.y, f.z, f.w};
  if (p.bias != nullptr) {
    const float4 b = __ldg(reinterpret_cast<const float4*>(p.bias + col));
    v[0] += b.x; v[1] += b.y; v[2] += b.z; v[3] += b.w;
  }
  if (p.z_out != nullptr)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.z_out) + at) =
        make_uint2(pack16(v[0], v[1], fp16), pack16(v[2], v[3], fp16));
  if (p.act != NVFP4MOE_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = act_value(v[i], p.act);
  }
  if (p.residual != nullptr) {
    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.residual) + at);
    const float2 f0 = unpack16(r.x, fp16), f1 = unpack16(r.y, fp16);
    v[0] += f0.x; v[1] += f0.y; v[2] += f1.x; v[3] += f1.y;
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
      make_uint2(pack16(v[0], v[1], fp16), pack16(v[2], v[3], fp16));
}

// 32 accumulator columns of this lane into the tile's column `lane`.
__device__ __forceinline__ void put_columns32(EpilogueTile& tile, const uint32_t* acc, int lane) {
  __syncwarp();   // the previous piece has been read
#pragma unroll
  for (int i = 0; i < 32; ++i) tile.v[i][lane] = __uint_as_float(acc[i]);
  __syncwarp();
}

// Stores `live` rows of the tile from out_row on, and of its columns (from col0 on) those below J,
// in 64-byte row pieces.
__device__ __forceinline__ void store_tile32(const EpilogueTile& tile, const MmArgs& p, int64_t out_row, int live,
                                             int col0, int lane) {
  const int c8 = (lane & 3) * 8, col = col0 + c8;
  if (col >= p.J) return;          // J is a multiple of 8
  float bias8[8];
  if (p.bias != nullptr) {
    const float4 b0 = __ldg(reinterpret_cast<const float4*>(p.bias + col));
    const float4 b1 = __ldg(reinterpret_cast<const float4*>(p.bias + col) + 1);
    bias8[0] = b0.x; bias8[1] = b0.y; bias8[2] = b0.z; bias8[3] = b0.w;
    bias8[4] = b1.x; bias8[5] = b1.y; bias8[6] = b1.z; bias8[7] = b1.w;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    if (r >= live) continue;
    const float4 x = *reinterpret_cast<const float4*>(&tile.v[r][c8]);
    const float4 y = *reinterpret_cast<const float4*>(&tile.v[r][c8 + 4]);
    float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    store8(p, v, bias8, (out_row + r) * (int64_t)p.J + col);
  }
}

}  // namespace nvfp4moe
