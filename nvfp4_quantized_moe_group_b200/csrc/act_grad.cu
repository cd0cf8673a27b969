// Gradient through the dense product's activation: dz = dy act'(z), rounded once to the operands'
// 16-bit type (dz feeds the two products of the backward pass, whose operands are 16-bit), and
// the bias gradient db = sum over rows of the unrounded FP32 dz.
//
// Memory bound: one pass over dy and z (16-byte loads, 8 columns a lane), dz written in the same
// pass.  A CTA owns 256 columns (32 lanes x 8) and a block of rows; its 8 warps take rows in turn
// and add their columns in registers, the warps' sums are added in shared memory and one row of
// partial sums per row block goes to the workspace; a second kernel adds those in a fixed order,
// so db does not depend on how the CTAs ran.  The first kernel of its call, it also resets the
// workspace's status word and work counters.
#include "activation.cuh"
#include "common.cuh"
#include "dense.h"
#include "kernels.h"

namespace nvfp4moe {

namespace {

constexpr int kThreads = 256;
constexpr int kCols = 256;               // columns of one CTA

template <int kAct>
__global__ void __launch_bounds__(kThreads)
act_grad_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ z, int64_t M, int N, int fp16,
                uint16_t* __restrict__ dz, float* __restrict__ partials, int64_t rows_per_block, WsHeader* hdr) {
  __shared__ float s_sum[8][kCols + 4];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    hdr->status = 0u;
    hdr->work[0] = hdr->work[1] = 0;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * kCols + lane * 8;
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_block;
  const int64_t r1 = r0 + rows_per_block < M ? r0 + rows_per_block : M;
  float sum[8] = {};
  if (col < N) {
#pragma unroll 4
    for (int64_t r = r0 + warp; r < r1; r += 8) {
      const int64_t at = r * N + col;
      const uint4 d4 = *reinterpret_cast<const uint4*>(dy + at);
      const uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w};
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack16(d[i], fp16 != 0);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
      if constexpr (kAct != NVFP4MOE_ACT_NONE) {
        const uint4 z4 = *reinterpret_cast<const uint4*>(z + at);
        const uint32_t zz[4] = {z4.x, z4.y, z4.z, z4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack16(zz[i], fp16 != 0);
          v[2 * i] *= act_slope<kAct>(f.x);
          v[2 * i + 1] *= act_slope<kAct>(f.y);
        }
        *reinterpret_cast<uint4*>(dz + at) =
            make_uint4(pack16(v[0], v[1], fp16 != 0), pack16(v[2], v[3], fp16 != 0), pack16(v[4], v[5], fp16 != 0),
                       pack16(v[6], v[7], fp16 != 0));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += v[i];
    }
  }
  if (partials == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) s_sum[warp][lane * 8 + i] = sum[i];
  __syncthreads();
  const int c = blockIdx.x * kCols + threadIdx.x;
  if (c < N) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += s_sum[i][threadIdx.x];
    partials[(int64_t)blockIdx.y * N + c] = t;
  }
}

// Adds n rows of partial sums: 32 columns a CTA, 8 slices of the rows side by side.
__global__ void __launch_bounds__(kThreads) sum_partials_kernel(const float* partials, int n, int N, float* out) {
  __shared__ float s[8][33];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float t = 0.0f;
  if (c < N) {
#pragma unroll 4
    for (int i = slice; i < n; i += 8) t += partials[(int64_t)i * N + c];
  }
  s[slice][lane] = t;
  __syncthreads();
  if (slice != 0 || c >= N) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) t += s[i][lane];
  out[c] = t;
}

}  // namespace

// Row blocks: enough CTAs for about 4 per SM of a B200, at least 32 rows each.
int act_grad_partials(int64_t M, int64_t N) {
  const int64_t col_blocks = (N + kCols - 1) / kCols;
  int64_t n = (4 * 148 + col_blocks - 1) / col_blocks;
  const int64_t most = (M + 31) / 32;
  if (n > most) n = most;
  return (int)(n < 1 ? 1 : n);
}

cudaError_t launch_act_grad(const void* dy, const void* z, int64_t M, int N, int act, bool fp16, void* dz, float* db,
                            float* partials, WsHeader* hdr, int* launches, cudaStream_t stream) {
  const int n = act_grad_partials(M, N);
  const int64_t rows = (M + n - 1) / n;
  cudaError_t e = cudaSuccess;
  with_act(act, [&](auto c) {
    e = launch_pdl(act_grad_kernel<decltype(c)::value>, dim3((N + kCols - 1) / kCols, n), dim3(kThreads), 0, stream,
                   static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(z), M, N, fp16 ? 1 : 0,
                   static_cast<uint16_t*>(dz), db != nullptr ? partials : nullptr, rows, hdr);
  });
  if (e != cudaSuccess) return e;
  ++*launches;
  if (db == nullptr) return cudaSuccess;
  e = launch_pdl(sum_partials_kernel, dim3((N + 31) / 32), dim3(kThreads), 0, stream,
                 (const float*)partials, n, N, db);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace nvfp4moe
