// Layer norm (and its RMS form) over the rows of a [rows][cols] matrix, forward and backward, with
// the reduction of the weight's and the bias's gradients over the rows.
//
//   forward   y = (x - mean) rstd gamma + beta,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   backward  xh = (x - mean) rstd,  g = dy gamma
//             dx = rstd (g - mean_j(g) - xh mean_j(g xh))
//             dgamma = sum_rows dy xh,  dbeta = sum_rows dy
// (RMS form: mean = 0 throughout, no mean_j(g) term, no beta.)
//
// All arithmetic is FP32; the variance is summed from the centred values, so a row's common offset
// costs no digits.  Both passes are memory bound (2 and 3 values moved per element).  A group of
// threads holds one row in registers, so x (and dy) are read from memory once; statistics are
// reduced by shuffles and, for groups of several warps, through shared memory.
//
// Backward: a persistent grid; each thread owns the same columns in every row of its group and
// adds their dgamma / dbeta terms in registers, so the column reduction costs no memory traffic
// per row; each CTA writes one row of partial sums and a second kernel adds those in a fixed
// order (the gradients do not depend on how the CTAs ran).  Rows too wide for that keep the
// column sums in shared memory and read x and dy a second time (from L2).
#include "activation.cuh"
#include "common.cuh"
#include "kernels.h"
#include "norm.h"

namespace nvfp4moe {

namespace {

constexpr int kNarrowCols = 8192;        // backward: widest row of the register kernel (512 threads x 16)

template <int kType> struct Elem { using T = uint16_t; };
template <> struct Elem<NVFP4MOE_FP32> { using T = float; };

template <int kBytes> struct VecOf;
template <> struct VecOf<16> { using T = uint4; };
template <> struct VecOf<8> { using T = uint2; };
template <> struct VecOf<4> { using T = uint32_t; };
template <> struct VecOf<2> { using T = uint16_t; };

template <int kType>
__device__ __forceinline__ float to_f32(typename Elem<kType>::T v) {
  if constexpr (kType == NVFP4MOE_FP32) return v;
  else if constexpr (kType == NVFP4MOE_FP16) return __half2float(__ushort_as_half(v));
  else return __uint_as_float((uint32_t)v << 16);
}

template <int kType>
__device__ __forceinline__ typename Elem<kType>::T from_f32(float v) {
  if constexpr (kType == NVFP4MOE_FP32) return v;
  else if constexpr (kType == NVFP4MOE_FP16) return __half_as_ushort(__float2half_rn(v));
  else return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// kVec consecutive elements (aligned to their size) <-> FP32.
template <int kType, int kVec>
__device__ __forceinline__ void load_vec(const void* base, int64_t at, float* v) {
  using T = typename Elem<kType>::T;
  using V = typename VecOf<kVec * (int)sizeof(T)>::T;
  const V raw = *reinterpret_cast<const V*>(static_cast<const T*>(base) + at);
  const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
  for (int i = 0; i < kVec; ++i) v[i] = to_f32<kType>(e[i]);
}

template <int kType, int kVec>
__device__ __forceinline__ void store_vec(void* base, int64_t at, const float* v) {
  using T = typename Elem<kType>::T;
  using V = typename VecOf<kVec * (int)sizeof(T)>::T;
  V raw;
  T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
  for (int i = 0; i < kVec; ++i) e[i] = from_f32<kType>(v[i]);
  *reinterpret_cast<V*>(static_cast<T*>(base) + at) = raw;
}

// Sums of kN values over the group's threads, for each group of the CTA (threadIdx.y).  Every
// thread of the CTA calls it.  s: kN * 32 floats per group.
template <int kN>
__device__ __forceinline__ void group_sum(float* v, float* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  s += threadIdx.y * kN * 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i * 32 + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    float t = lane < warps ? s[i * 32 + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    v[i] = t;
  }
}

// One row per group of blockDim.x threads, blockDim.y groups; kPer elements a thread in vectors
// of kVec: thread t holds vectors t, t + blockDim.x, ...
template <int kType, int kVec, int kPer>
__global__ void __launch_bounds__(1024) norm_forward_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kVecs = kPer / kVec;
  __shared__ float s_red[8 * 32];
  pdl_wait();
  pdl_trigger();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < a.rows;
  const int64_t base = row * a.cols;
  float v[kVecs][kVec];
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const int c = (k * blockDim.x + threadIdx.x) * kVec;
    if (live && c < a.cols) {
      load_vec<kType, kVec>(a.x, base + c, v[k]);
#pragma unroll
      for (int i = 0; i < kVec; ++i) sum += v[k][i];
    }
  }
  float mean = 0.0f;
  if (!a.rms) {
    group_sum<1>(&sum, s_red);
    mean = sum / (float)a.cols;
  }
  float sq = 0.0f;
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const int c = (k * blockDim.x + threadIdx.x) * kVec;
    if (live && c < a.cols) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        v[k][i] -= mean;
        sq = fmaf(v[k][i], v[k][i], sq);
      }
    }
  }
  group_sum<1>(&sq, s_red);
  const float rstd = 1.0f / sqrtf(sq / (float)a.cols + a.eps);
  if (!live) return;
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const int c = (k * blockDim.x + threadIdx.x) * kVec;
    if (c >= a.cols) continue;
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[k][i] *= rstd;
    if (a.gamma != nullptr) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[k][i] *= __ldg(a.gamma + c + i);
    }
    if (a.beta != nullptr) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[k][i] += __ldg(a.beta + c + i);
    }
    store_vec<kType, kVec>(a.y, base + c, v[k]);
  }
}

// Register kernel of the backward pass: blockDim.y row groups per CTA, rows in turn.
template <int kType, int kVec, int kPer>
__global__ void __launch_bounds__(512) norm_backward_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kVecs = kPer / kVec;
  extern __shared__ float s_dyn[];       // 2 * cols when the CTA has several groups
  __shared__ float s_red[8 * 2 * 32];
  pdl_wait();
  pdl_trigger();
  float dg[kVecs][kVec] = {}, db[kVecs][kVec] = {}, gam[kVecs][kVec];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const int c = (k * blockDim.x + threadIdx.x) * kVec;
#pragma unroll
    for (int i = 0; i < kVec; ++i) gam[k][i] = a.gamma != nullptr && c < a.cols ? __ldg(a.gamma + c + i) : 1.0f;
  }
  const float inv_cols = 1.0f / (float)a.cols;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  for (int64_t row0 = (int64_t)blockIdx.x * blockDim.y; row0 < a.rows; row0 += step) {
    const int64_t row = row0 + threadIdx.y;
    const bool live = row < a.rows;
    const int64_t base = row * a.cols;
    const float mean = live && !a.rms ? a.mean[row] : 0.0f;
    const float rstd = live ? a.rstd[row] : 0.0f;
    float x[kVecs][kVec], dy[kVecs][kVec];
    float sums[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int c = (k * blockDim.x + threadIdx.x) * kVec;
      if (live && c < a.cols) {
        load_vec<kType, kVec>(a.x, base + c, x[k]);
        load_vec<kType, kVec>(a.dy, base + c, dy[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int c = (k * blockDim.x + threadIdx.x) * kVec;
      if (live && c < a.cols) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          x[k][i] = (x[k][i] - mean) * rstd;
          dg[k][i] = fmaf(dy[k][i], x[k][i], dg[k][i]);
          db[k][i] += dy[k][i];
          dy[k][i] *= gam[k][i];
          sums[0] += dy[k][i];
          sums[1] = fmaf(dy[k][i], x[k][i], sums[1]);
        }
      }
    }
    group_sum<2>(sums, s_red);
    const float mg = a.rms ? 0.0f : sums[0] * inv_cols;
    const float mgx = sums[1] * inv_cols;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int c = (k * blockDim.x + threadIdx.x) * kVec;
      if (live && c < a.cols) {
        float o[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) o[i] = rstd * (dy[k][i] - mg - x[k][i] * mgx);
        store_vec<kType, kVec>(a.dx, base + c, o);
      }
    }
  }
  if (a.partials == nullptr) return;
  float* part = a.partials + (int64_t)blockIdx.x * 2 * a.cols;
  if (blockDim.y == 1) {
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int c = (k * blockDim.x + threadIdx.x) * kVec;
      if (c < a.cols)
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          part[c + i] = dg[k][i];
          part[a.cols + c + i] = db[k][i];
        }
    }
    return;
  }
  // the groups add their columns one after the other
  for (int g = 0; g < (int)blockDim.y; ++g) {
    if ((int)threadIdx.y == g) {
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const int c = (k * blockDim.x + threadIdx.x) * kVec;
        if (c < a.cols)
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            s_dyn[c + i] = (g != 0 ? s_dyn[c + i] : 0.0f) + dg[k][i];
            s_dyn[a.cols + c + i] = (g != 0 ? s_dyn[a.cols + c + i] : 0.0f) + db[k][i];
          }
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < 2 * a.cols; c += blockDim.x * blockDim.y) part[c] = s_dyn[c];
}

// Wide rows: 1024 threads a row, x and dy read twice, the column sums in shared memory (each
// thread adds only into its own columns).
template <int kType, int kVec>
__global__ void __launch_bounds__(1024) norm_backward_wide_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ float s_dyn[];       // [2][cols]
  __shared__ float s_red[2 * 32];
  pdl_wait();
  pdl_trigger();
  const int step = blockDim.x * kVec;
  for (int c = threadIdx.x; c < 2 * a.cols; c += blockDim.x) s_dyn[c] = 0.0f;
  __syncthreads();
  const float inv_cols = 1.0f / (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t base = row * a.cols;
    const float mean = a.rms ? 0.0f : a.mean[row];
    const float rstd = a.rstd[row];
    float sums[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x * kVec; c < a.cols; c += step) {
      float x[kVec], dy[kVec];
      load_vec<kType, kVec>(a.x, base + c, x);
      load_vec<kType, kVec>(a.dy, base + c, dy);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float xh = (x[i] - mean) * rstd;
        s_dyn[c + i] = fmaf(dy[i], xh, s_dyn[c + i]);
        s_dyn[a.cols + c + i] += dy[i];
        const float g = a.gamma != nullptr ? dy[i] * __ldg(a.gamma + c + i) : dy[i];
        sums[0] += g;
        sums[1] = fmaf(g, xh, sums[1]);
      }
    }
    group_sum<2>(sums, s_red);
    const float mg = a.rms ? 0.0f : sums[0] * inv_cols;
    const float mgx = sums[1] * inv_cols;
    for (int c = threadIdx.x * kVec; c < a.cols; c += step) {
      float x[kVec], dy[kVec], o[kVec];
      load_vec<kType, kVec>(a.x, base + c, x);
      load_vec<kType, kVec>(a.dy, base + c, dy);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float xh = (x[i] - mean) * rstd;
        const float g = a.gamma != nullptr ? dy[i] * __ldg(a.gamma + c + i) : dy[i];
        o[i] = rstd * (g - mg - xh * mgx);
      }
      store_vec<kType, kVec>(a.dx, base + c, o);
    }
  }
  __syncthreads();
  if (a.partials == nullptr) return;
  float* part = a.partials + (int64_t)blockIdx.x * 2 * a.cols;
  for (int c = threadIdx.x; c < 2 * a.cols; c += blockDim.x) part[c] = s_dyn[c];
}

// Adds the CTAs' partial sums: 32 columns a CTA, 8 slices of the parts side by side.
__global__ void __launch_bounds__(256) norm_param_sum_kernel(const float* partials, int parts, int cols, float* dgamma,
                                                             float* dbeta) {
  __shared__ float s[8][33];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;              // column of [dgamma | dbeta]
  float t = 0.0f;
  if (c < 2 * cols)
    for (int i = slice; i < parts; i += 8) t += partials[(int64_t)i * 2 * cols + c];
  s[slice][lane] = t;
  __syncthreads();
  if (slice != 0 || c >= 2 * cols) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) t += s[i][lane];
  if (c < cols) {
    if (dgamma != nullptr) dgamma[c] = t;
  } else if (dbeta != nullptr) {
    dbeta[c - cols] = t;
  }
}

// Threads of a row group for `per` elements a thread, and row groups per CTA.
dim3 group_shape(int cols, int per, int max_threads) {
  const int threads = ((cols + per - 1) / per + 31) / 32 * 32;
  int groups = threads < 128 ? 256 / threads : 1;
  if (groups > 8) groups = 8;
  if (threads * groups > max_threads) groups = 1;
  return dim3(threads, groups);
}

template <int kType, int kVec>
cudaError_t forward_vec(const NormArgs& a, cudaStream_t stream) {
  auto go = [&](auto kernel, int per) {
    const dim3 block = group_shape(a.cols, per, 1024);
    return launch_pdl(kernel, dim3((unsigned)((a.rows + block.y - 1) / block.y)), block, 0, stream, a);
  };
  if (a.cols <= 2048) return go(norm_forward_kernel<kType, kVec, 8>, 8);
  if (a.cols <= 16384) return go(norm_forward_kernel<kType, kVec, 16>, 16);
  return go(norm_forward_kernel<kType, kVec, 32>, 32);
}

int backward_ctas(int64_t rows, int cols) {
  const bool narrow = cols <= kNarrowCols;
  const int groups = narrow ? (int)group_shape(cols, cols <= 2048 ? 8 : 16, 512).y : 1;
  const int64_t ctas = (rows + groups - 1) / groups;
  const int64_t most = (int64_t)(narrow ? 4 : 1) * 148;
  return (int)(ctas < most ? ctas : most);
}

template <int kType, int kVec>
cudaError_t backward_vec(const NormArgs& a, int ctas, cudaStream_t stream) {
  if (a.cols > kNarrowCols) {
    const size_t smem = (size_t)2 * a.cols * sizeof(float);
    auto kernel = norm_backward_wide_kernel<kType, kVec>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(ctas), dim3(1024), smem, stream, a);
  }
  auto go = [&](auto kernel, int per) {
    const dim3 block = group_shape(a.cols, per, 512);
    return launch_pdl(kernel, dim3(ctas), block, block.y > 1 ? (size_t)2 * a.cols * sizeof(float) : 0, stream, a);
  };
  if (a.cols <= 2048) return go(norm_backward_kernel<kType, kVec, 8>, 8);
  return go(norm_backward_kernel<kType, kVec, 16>, 16);
}


template <int kType>
cudaError_t forward_type(const NormArgs& a, cudaStream_t stream) {
  constexpr int kWide = kType == NVFP4MOE_FP32 ? 4 : 8;
  if (a.cols % kWide == 0) return forward_vec<kType, kWide>(a, stream);
  if (a.cols % 2 == 0) return forward_vec<kType, 2>(a, stream);
  return forward_vec<kType, 1>(a, stream);
}

template <int kType>
cudaError_t backward_type(const NormArgs& a, int ctas, cudaStream_t stream) {
  constexpr int kWide = kType == NVFP4MOE_FP32 ? 4 : 8;
  if (a.cols % kWide == 0) return backward_vec<kType, kWide>(a, ctas, stream);
  if (a.cols % 2 == 0) return backward_vec<kType, 2>(a, ctas, stream);
  return backward_vec<kType, 1>(a, ctas, stream);
}

}  // namespace

int norm_backward_parts(int64_t rows, int cols) { return backward_ctas(rows, cols); }

cudaError_t launch_norm_forward(const NormArgs& a, int* launches, cudaStream_t stream) {
  cudaError_t e;
  switch (a.dtype) {
    case NVFP4MOE_BF16: e = forward_type<NVFP4MOE_BF16>(a, stream); break;
    case NVFP4MOE_FP16: e = forward_type<NVFP4MOE_FP16>(a, stream); break;
    default: e = forward_type<NVFP4MOE_FP32>(a, stream);
  }
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_norm_backward(const NormArgs& a, int* launches, cudaStream_t stream) {
  const int ctas = backward_ctas(a.rows, a.cols);
  cudaError_t e;
  switch (a.dtype) {
    case NVFP4MOE_BF16: e = backward_type<NVFP4MOE_BF16>(a, ctas, stream); break;
    case NVFP4MOE_FP16: e = backward_type<NVFP4MOE_FP16>(a, ctas, stream); break;
    default: e = backward_type<NVFP4MOE_FP32>(a, ctas, stream);
  }
  if (e != cudaSuccess) return e;
  ++*launches;
  if (a.partials == nullptr) return cudaSuccess;
  e = launch_pdl(norm_param_sum_kernel, dim3((2 * a.cols + 31) / 32), dim3(256), 0, stream, (const float*)a.partials,
                 ctas, a.cols, a.dgamma, a.dbeta);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace nvfp4moe
