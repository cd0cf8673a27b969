// Layer norm (and its RMS form) over the rows of a [rows][cols] matrix, forward and backward, with
// the reduction of the weight's and the bias's gradients over the rows.
//
//   forward   y = (x - mean) rstd gamma + beta,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   backward  xh = (x - mean) rstd,  g = dy gamma
//             dx = rstd (g - mean_j(g) - xh mean_j(g xh))
//             dgamma = sum_rows dy xh,  dbeta = sum_rows dy
// (RMS form: mean = 0 throughout, no mean_j(g) term, no beta.)
//
// All arithmetic is FP32; the variance is summed from the centred values, so a row's common offset costs
// digits in the mean only (a few units of 2^-24 of the offset).  Both passes are memory bound (2 and 3 values moved
// per element).
//
// One persistent CTA per SM holds several groups of threads; each group takes rows in turn, each
// thread its own 16-byte vectors of them (32 elements a thread, so that the reductions' fixed cost
// is spread over many; the kernels are close to bound by instruction issue).  A thread copies its own
// vectors of the coming rows into shared memory with cp.async (no other thread reads them, so no
// barrier), rows ahead, so loads stay in flight across the reductions; the other groups' work
// covers a group's own latency.  Row sums are reduced by shuffles and, for groups of several warps,
// through shared memory with one named barrier a reduction (every thread adds the warps' sums itself,
// in buffers that alternate).  The parameters lie in shared memory once for all groups.
//
// Row lengths that are no multiple of a vector: a row then starts `lead` elements into an aligned
// vector.  lead depends on the row's index modulo the vector length only, and a CTA takes rows of one
// residue modulo 8, so a thread's columns stay the same through all its rows: column sums stay in
// registers, the parameters are staged shifted by lead, the first and last vector of a row are masked,
// and all other accesses are whole vectors.
//
// Backward: each thread adds its columns' dgamma / dbeta terms in registers, so the column
// reduction costs no memory traffic per row; each CTA adds its groups' sums, writes one row of partial
// sums, and a second kernel adds those in a fixed order (the gradients do not depend on how the CTAs
// ran).  Rows too wide for that keep the column sums in shared memory and read x and dy a second time
// (from L2).
//
// Measured in a replayed graph: 32768 x 5120 BF16 forward 137 us (4.9 TB/s), backward 197 us (5.1 TB/s; called 217 to 222);
// 8191 x 2571 FP32 forward 35 to 36 us (4.8 TB/s); 16 x 5120 forward 3.1 us (called 12).
#include "activation.cuh"
#include "common.cuh"
#include "kernels.h"
#include "norm.h"

namespace nvfp4moe {

namespace {

template <int kType> struct Elem { using T = uint16_t; };
template <> struct Elem<NVFP4MOE_FP32> { using T = float; };

template <int kType>
__device__ __forceinline__ float to_f32(typename Elem<kType>::T v) {
  if constexpr (kType == NVFP4MOE_FP32) return v;
  else if constexpr (kType == NVFP4MOE_FP16) return __half2float(__ushort_as_half(v));
  else return __uint_as_float((uint32_t)v << 16);
}

// Sums of kN values over the CTA's threads (one group), in every thread.  s: kN * 32 floats that no
// other thread still reads (callers alternate two buffers).
template <int kN>
__device__ __forceinline__ void group_sum(float* v, float* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i * 32 + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = lane < warps ? s[i * 32 + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// Sums of kN values over one group of kG threads, in every thread: the warps' sums are added one after
// the other, their loads independent.  s: kN * kG / 32 floats that no thread of the group still reads.
template <int kN, int kG>
__device__ __forceinline__ void ring_sum(float* v, float* s, int group) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (kG > 32) {
    const int warp = (threadIdx.x % kG) >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < kN; ++i) s[kN * warp + i] = v[i];
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kG) : "memory");
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = s[i];
#pragma unroll
    for (int j = 1; j < kG / 32; ++j)
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] += s[kN * j + i];
  }
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A thread's vectors of its rows: vector k covers columns col(k) .. col(k) + kVec - 1.  kAligned: the
// row length is a multiple of kVec, so every vector with a column in the row lies in it whole.
template <int kType, bool kAligned, int kG, int kPer>
struct Columns {
  static constexpr int kVec = 16 / (int)sizeof(typename Elem<kType>::T);
  static constexpr int kVecs = kPer / kVec;
  static constexpr int kParamFloats = kG * kPer;       // a parameter array in shared memory
  int cols, lead, col0;
  __device__ __forceinline__ Columns(const NormArgs& a, int64_t first_row)
      : cols(a.cols), lead(kAligned ? 0 : (int)((first_row * a.cols) % kVec)) {
    col0 = (int)(threadIdx.x % kG) * kVec - lead;
  }
  // The first row of group g of this CTA and the step to its next one (see lead above).
  static __device__ __forceinline__ int64_t first_row(int groups, int g) {
    if (kAligned) return (int64_t)blockIdx.x * groups + g;
    return 8 * ((int64_t)(blockIdx.x >> 3) * groups + g) + (blockIdx.x & 7);
  }
  __device__ __forceinline__ int col(int k) const { return col0 + k * kG * kVec; }
  __device__ __forceinline__ bool some(int k) const { return col(k) < cols; }
  __device__ __forceinline__ bool whole(int k) const { return kAligned || (col(k) >= 0 && col(k) + kVec <= cols); }
  __device__ __forceinline__ bool has(int k, int i) const { return col(k) + i >= 0 && col(k) + i < cols; }
  // Parameters shifted by lead, so that a thread's vector is aligned; `none` outside the row.
  __device__ __forceinline__ void stage_params(float* s, const float* p, float none) const {
    for (int j = threadIdx.x; j < kParamFloats; j += blockDim.x) {
      const int c = j - lead;
      s[j] = p != nullptr && c >= 0 && c < cols ? __ldg(p + c) : none;
    }
  }
  __device__ __forceinline__ void params(const float* s, int k, float* v) const {
#pragma unroll
    for (int i = 0; i < kVec / 4; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(s + col(k) + lead + 4 * i);
      v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
    }
  }
  // The same straight from global memory (`vec`: p is 16-byte aligned).  A vector that starts shift
  // floats into an aligned one takes one 16-byte load more; shift is the same for the whole CTA.
  __device__ __forceinline__ void params_global(const float* p, bool vec, float none, int k, float* v) const {
    const int c = col(k);
    if (p == nullptr) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = none;
    } else if (kAligned ? vec : vec && c >= 0 && c + kVec + 4 <= cols) {
      const int shift = kAligned ? 0 : (c & 3);
      const float4* at = reinterpret_cast<const float4*>(p + c - shift);
      float f[kVec + 4];
#pragma unroll
      for (int i = 0; i < kVec / 4; ++i) {
        const float4 q = __ldg(at + i);
        f[4 * i] = q.x; f[4 * i + 1] = q.y; f[4 * i + 2] = q.z; f[4 * i + 3] = q.w;
      }
      if (!kAligned && shift != 0) {
        const float4 q = __ldg(at + kVec / 4);
        f[kVec] = q.x; f[kVec + 1] = q.y; f[kVec + 2] = q.z; f[kVec + 3] = q.w;
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = shift == 1 ? f[i + 1] : shift == 2 ? f[i + 2] : f[i + 3];
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = f[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = has(k, i) ? __ldg(p + c + i) : none;
    }
  }
  // Starts the copy of vector k of a row (the elements in front of the row are the previous row's;
  // none behind it are read).
  __device__ __forceinline__ void fetch(void* dst, const void* base, int64_t row, int k) const {
    const int c = col(k), left = cols - c;
    using T = typename Elem<kType>::T;
    cp_async16(dst, static_cast<const T*>(base) + row * cols + c,
               kAligned || left >= kVec ? 16 : left * (int)sizeof(T));
  }
  // Only a row's first vector (k = 0 of the first thread) has elements in front of the row, only its last
  // one elements behind it.
  __device__ __forceinline__ bool head(int k) const { return !kAligned && k == 0 && col0 < 0; }
  __device__ __forceinline__ bool tail(int k) const { return !kAligned && col(k) + kVec > cols; }
  // The values of one vector; 0 outside the row (the copy has filled zeros behind it).
  __device__ __forceinline__ void values(const uint4& raw, int k, float* v) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kType == NVFP4MOE_FP32) {
        v[i] = __uint_as_float(w[i]);
      } else {
        const float2 f = unpack16(w[i], kType == NVFP4MOE_FP16);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
    clear_head(k, v);
  }
  __device__ __forceinline__ void clear_head(int k, float* v) const {
    if (head(k)) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = i < lead ? 0.0f : v[i];
    }
  }
  __device__ __forceinline__ void clear(int k, float* v) const {
    clear_head(k, v);
    if (tail(k)) {
      const int left = cols - col(k);
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = i < left ? v[i] : 0.0f;
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t row, int k, const float* v) const {
    using T = typename Elem<kType>::T;
    T* at = static_cast<T*>(base) + row * cols + col(k);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kType == NVFP4MOE_FP32) w[i] = __float_as_uint(v[i]);
      else w[i] = pack16(v[2 * i], v[2 * i + 1], kType == NVFP4MOE_FP16);
    }
    if (!head(k) && !tail(k)) {
      *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      const int from = head(k) ? lead : 0, to = tail(k) ? cols - col(k) : kVec;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        if (i < from || i >= to) continue;
        if constexpr (kType == NVFP4MOE_FP32) at[i] = v[i];
        else at[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
      }
    }
  }
};

// Shared memory of the ring kernels: kGroups groups of kG threads with rings of rows, and the
// parameters (kParams arrays, 0: too wide, they are read from global memory).
constexpr size_t kNormSmem = 222 * 1024;
template <int kType, bool kAligned, int kG, int kPer, int kGroups, int kStreams, int kParams>
struct Ring {
  using Cols = Columns<kType, kAligned, kG, kPer>;
  static constexpr size_t kParamBytes = (size_t)kParams * ((Cols::kParamFloats * 4 + 15) / 16 * 16);
  static constexpr size_t kRowBytes = (size_t)kGroups * kG * kPer * sizeof(typename Elem<kType>::T) * kStreams;
  static constexpr int kFit = (int)((kNormSmem - kParamBytes) / kRowBytes);
  static constexpr int kRows = kFit > 4 ? 4 : kFit;
  static constexpr size_t kBytes = kParamBytes + kRows * kRowBytes;
  static_assert(kRows >= 1, "a row of every group fits shared memory");
};

// kR rows at a time per group: the parameters' reads and the barriers serve all of them.
template <int kType, bool kAligned, int kG, int kPer, int kGroups, int kR, int kParams>
__global__ void __launch_bounds__(kG * kGroups, 1) norm_forward_kernel(const __grid_constant__ NormArgs a) {
  using R = Ring<kType, kAligned, kG, kPer, kGroups, kR, kParams>;
  using Cols = typename R::Cols;
  constexpr int kVec = Cols::kVec, kVecs = Cols::kVecs, kRing = R::kRows, kThreads = kG * kGroups;
  extern __shared__ __align__(16) uint8_t s_dyn[];
  float* s_gamma = reinterpret_cast<float*>(s_dyn);
  float* s_beta = reinterpret_cast<float*>(s_dyn + R::kParamBytes / 2);
  uint4* s_ring = reinterpret_cast<uint4*>(s_dyn + R::kParamBytes) + threadIdx.x;    // [kRing][kR][kVecs][threads]
  __shared__ float s_red[kGroups][2][kR * (kG / 32)];
  pdl_wait();
  pdl_trigger();
  const int group = threadIdx.x / kG;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  int64_t row = Cols::first_row(kGroups, group);
  const Cols c(a, row);
  auto slot = [&](int at, int r, int k) { return s_ring + ((at * kR + r) * kVecs + k) * kThreads; };
  auto fetch = [&](int64_t row0, int at) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int64_t from = row0 + r * step;
      if (from < a.rows) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
          if (c.some(k)) c.fetch(slot(at, r, k), a.x, from, k);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) fetch(row + i * kR * step, i);
  const bool affine = a.gamma != nullptr || a.beta != nullptr;
  const bool vec_g = (reinterpret_cast<uintptr_t>(a.gamma) & 15) == 0;
  const bool vec_b = (reinterpret_cast<uintptr_t>(a.beta) & 15) == 0;
  if (kParams > 0 && affine) {
    c.stage_params(s_gamma, a.gamma, 1.0f);
    c.stage_params(s_beta, a.beta, 0.0f);
    __syncthreads();
  }
  const float inv_cols = 1.0f / (float)a.cols;
  int at = 0, turn = 0;
  for (; row < a.rows; row += kR * step) {
    fetch(row + (kRing - 1) * kR * step, at == 0 ? kRing - 1 : at - 1);
    cp_async_wait<kRing - 1>();
    float v[kR][kVecs][kVec], mean[kR], sq[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const bool live = r == 0 || row + r * step < a.rows;
      mean[r] = 0.0f;
#pragma unroll
      for (int k = 0; k < kVecs; ++k)
        if (live && c.some(k)) {
          c.values(*slot(at, r, k), k, v[r][k]);
#pragma unroll
          for (int i = 0; i < kVec; ++i) mean[r] += v[r][k][i];
        }
    }
    if (!a.rms) {
      ring_sum<kR, kG>(mean, s_red[group][0], group);
#pragma unroll
      for (int r = 0; r < kR; ++r) mean[r] *= inv_cols;
    } else {
#pragma unroll
      for (int r = 0; r < kR; ++r) mean[r] = 0.0f;
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const bool live = r == 0 || row + r * step < a.rows;
      sq[r] = 0.0f;
#pragma unroll
      for (int k = 0; k < kVecs; ++k)
        if (live && c.some(k)) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) v[r][k][i] -= mean[r];
          c.clear(k, v[r][k]);
#pragma unroll
          for (int i = 0; i < kVec; ++i) sq[r] = fmaf(v[r][k][i], v[r][k][i], sq[r]);
        }
    }
    ring_sum<kR, kG>(sq, s_red[group][a.rms ? turn : 1], group);
    float rstd[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      rstd[r] = rsqrtf(fmaf(sq[r], inv_cols, a.eps));
      if (threadIdx.x % kG == 0 && (r == 0 || row + r * step < a.rows)) {
        if (a.mean != nullptr) a.mean[row + r * step] = mean[r];
        if (a.rstd != nullptr) a.rstd[row + r * step] = rstd[r];
      }
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      if (c.some(k)) {
        float g[kVec], b[kVec];
        if (affine) {
          if (kParams > 0) {
            c.params(s_gamma, k, g);
            c.params(s_beta, k, b);
          } else {
            c.params_global(a.gamma, vec_g, 1.0f, k, g);
            c.params_global(a.beta, vec_b, 0.0f, k, b);
          }
        }
#pragma unroll
        for (int r = 0; r < kR; ++r)
          if (r == 0 || row + r * step < a.rows) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[r][k][i] *= rstd[r];
            if (affine) {
#pragma unroll
              for (int i = 0; i < kVec; ++i) v[r][k][i] = fmaf(v[r][k][i], g[i], b[i]);
            }
            c.store(a.y, row + r * step, k, v[r][k]);
          }
      }
    at = at == kRing - 1 ? 0 : at + 1;
    turn ^= 1;
  }
}

// Backward: x and dy in the ring, read twice from there (for the row's sums, then for dx).
template <int kType, bool kAligned, int kG, int kPer, int kGroups, int kParams>
__global__ void __launch_bounds__(kG * kGroups, 1) norm_backward_kernel(const __grid_constant__ NormArgs a) {
  using R = Ring<kType, kAligned, kG, kPer, kGroups, 2, kParams>;
  using Cols = typename R::Cols;
  constexpr int kVec = Cols::kVec, kVecs = Cols::kVecs, kRing = R::kRows, kThreads = kG * kGroups;
  extern __shared__ __align__(16) uint8_t s_dyn[];
  float* s_gamma = reinterpret_cast<float*>(s_dyn);
  uint4* s_ring = reinterpret_cast<uint4*>(s_dyn + R::kParamBytes) + threadIdx.x;    // [kRing][2][kVecs][threads]
  __shared__ float s_red[kGroups][2][2 * (kG / 32)];
  pdl_wait();
  pdl_trigger();
  const int group = threadIdx.x / kG;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  int64_t row = Cols::first_row(kGroups, group);
  const Cols c(a, row);
  auto slot = [&](int at, int which, int k) { return s_ring + ((at * 2 + which) * kVecs + k) * kThreads; };
  auto fetch = [&](int64_t r, int at) {
    if (r < a.rows) {
#pragma unroll
      for (int k = 0; k < kVecs; ++k)
        if (c.some(k)) {
          c.fetch(slot(at, 0, k), a.x, r, k);
          c.fetch(slot(at, 1, k), a.dy, r, k);
        }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) fetch(row + i * step, i);
  const bool has_gamma = a.gamma != nullptr;
  const bool vec_g = (reinterpret_cast<uintptr_t>(a.gamma) & 15) == 0;
  if (kParams > 0 && has_gamma) {
    c.stage_params(s_gamma, a.gamma, 1.0f);
    __syncthreads();
  }
  auto gammas = [&](int k, float* g) {
    if (kParams > 0 && has_gamma) c.params(s_gamma, k, g);
    else c.params_global(a.gamma, vec_g, 1.0f, k, g);
  };
  float dg[kVecs][kVec] = {}, db[kVecs][kVec] = {};
  const float inv_cols = 1.0f / (float)a.cols;
  float mean_next = 0.0f, rstd_next = 0.0f;
  auto fetch_stats = [&](int64_t r) {
    if (r < a.rows) {
      mean_next = a.rms ? 0.0f : __ldg(a.mean + r);
      rstd_next = __ldg(a.rstd + r);
    }
  };
  fetch_stats(row);
  int at = 0, turn = 0;
  for (; row < a.rows; row += step) {
    const float mean = mean_next, rstd = rstd_next;
    fetch(row + (kRing - 1) * step, at == 0 ? kRing - 1 : at - 1);
    fetch_stats(row + step);
    cp_async_wait<kRing - 1>();
    // with t = x - mean and u = dy t: dgamma += u rstd, and rstd leaves the row's sum of u gamma
    float sums[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      if (c.some(k)) {
        float x[kVec], d[kVec], g[kVec];
        c.values(*slot(at, 0, k), k, x);
        c.values(*slot(at, 1, k), k, d);
        gammas(k, g);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float u = d[i] * (x[i] - mean);
          dg[k][i] = fmaf(u, rstd, dg[k][i]);
          db[k][i] += d[i];
          sums[0] = fmaf(d[i], g[i], sums[0]);
          sums[1] = fmaf(u, g[i], sums[1]);
        }
      }
    ring_sum<2, kG>(sums, s_red[group][turn], group);
    // dx = rstd g - rstd mean_j(g) - t rstd^2 mean_j(g xh)
    const float shift = a.rms ? 0.0f : -sums[0] * inv_cols * rstd;
    const float slope = -(sums[1] * inv_cols * rstd) * (rstd * rstd);
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      if (c.some(k)) {
        float x[kVec], d[kVec], g[kVec];
        c.values(*slot(at, 0, k), k, x);
        c.values(*slot(at, 1, k), k, d);
        gammas(k, g);
#pragma unroll
        for (int i = 0; i < kVec; ++i) d[i] = fmaf(d[i] * g[i], rstd, fmaf(x[i] - mean, slope, shift));
        c.store(a.dx, row, k, d);
      }
    at = at == kRing - 1 ? 0 : at + 1;
    turn ^= 1;
  }
  if (a.partials == nullptr) return;
  // The groups' sums side by side in shared memory that is no longer used, by place in the vectors (column
  // + lead, which all rows of a CTA share), added in group order.  From there whole lines leave: stored
  // by the threads that hold them, 8 columns apart, 21 rows x 12146 took 21.8 us.
  cp_async_wait<0>();
  __syncthreads();
  constexpr int kPlaces = kG * kPer;
  float* s_sum = reinterpret_cast<float*>(s_dyn);      // [kGroups][2][kPlaces]
  static_assert(R::kBytes >= (size_t)kGroups * 2 * kPlaces * sizeof(float), "the column sums fit the rings");
  float* mine = s_sum + (size_t)group * 2 * kPlaces;
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
#pragma unroll
    for (int i = 0; i < kVec; i += 4) {
      float* to = mine + (k * kG + threadIdx.x % kG) * kVec + i;
      *reinterpret_cast<float4*>(to) = make_float4(dg[k][i], dg[k][i + 1], dg[k][i + 2], dg[k][i + 3]);
      *reinterpret_cast<float4*>(to + kPlaces) = make_float4(db[k][i], db[k][i + 1], db[k][i + 2], db[k][i + 3]);
    }
  __syncthreads();
  float* part = a.partials + (int64_t)blockIdx.x * 2 * a.cols;
  for (int i = threadIdx.x; i < 2 * a.cols; i += kThreads) {
    const float* from = s_sum + (i < a.cols ? i : i - a.cols + kPlaces) + c.lead;
    float sum = *from;
    for (int g = 1; g < kGroups; ++g) sum += from[(size_t)g * 2 * kPlaces];
    part[i] = sum;
  }
}

// Wide rows: 1024 threads a row, x and dy read twice, the column sums in shared memory, each thread's
// own (16 bytes a thread and access, so no bank conflicts).
template <int kType, bool kAligned>
__global__ void __launch_bounds__(1024) norm_backward_wide_kernel(const __grid_constant__ NormArgs a, int n_vecs) {
  using Cols = Columns<kType, kAligned, 1024, 32>;
  constexpr int kVec = Cols::kVec, kQuads = kVec / 4;
  extern __shared__ float4 s_acc[];      // [2: dgamma, dbeta][kQuads][n_vecs]
  __shared__ float s_red[2][2 * 32];
  pdl_wait();
  pdl_trigger();
  const int64_t step = gridDim.x;
  int64_t row = Cols::first_row(1, 0);
  const Cols c(a, row);
  const bool vec_g = (reinterpret_cast<uintptr_t>(a.gamma) & 15) == 0;
  for (int j = threadIdx.x; j < 2 * kQuads * n_vecs; j += 1024) s_acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  const float inv_cols = 1.0f / (float)a.cols;
  auto load = [&](const void* base, int64_t r, int k, float* v) {
    using T = typename Elem<kType>::T;
    const T* at = static_cast<const T*>(base) + r * a.cols + c.col(k);
    if (c.whole(k)) {
      c.values(__ldg(reinterpret_cast<const uint4*>(at)), k, v);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = c.has(k, i) ? to_f32<kType>(at[i]) : 0.0f;
    }
  };
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    const float mean = a.rms ? 0.0f : __ldg(a.mean + row);
    const float rstd = __ldg(a.rstd + row);
    float sums[2] = {0.0f, 0.0f};
#pragma unroll 2
    for (int k = 0; c.some(k); ++k) {
      float x[kVec], d[kVec], g[kVec];
      load(a.x, row, k, x);
      load(a.dy, row, k, d);
      c.params_global(a.gamma, vec_g, 1.0f, k, g);
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        float4* pg = s_acc + q * n_vecs + k * 1024 + threadIdx.x;
        float4* pb = pg + kQuads * n_vecs;
        float4 vg = *pg, vb = *pb;
        float* eg = &vg.x;
        float* eb = &vb.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float dv = d[4 * q + i], u = dv * (x[4 * q + i] - mean);
          eg[i] = fmaf(u, rstd, eg[i]);
          eb[i] += dv;
          sums[0] = fmaf(dv, g[4 * q + i], sums[0]);
          sums[1] = fmaf(u, g[4 * q + i], sums[1]);
        }
        *pg = vg;
        *pb = vb;
      }
    }
    group_sum<2>(sums, s_red[turn]);
    const float shift = a.rms ? 0.0f : -sums[0] * inv_cols * rstd;
    const float slope = -(sums[1] * inv_cols * rstd) * (rstd * rstd);
#pragma unroll 2
    for (int k = 0; c.some(k); ++k) {
      float x[kVec], d[kVec], g[kVec];
      load(a.x, row, k, x);
      load(a.dy, row, k, d);
      c.params_global(a.gamma, vec_g, 1.0f, k, g);
#pragma unroll
      for (int i = 0; i < kVec; ++i) d[i] = fmaf(d[i] * g[i], rstd, fmaf(x[i] - mean, slope, shift));
      c.store(a.dx, row, k, d);
    }
  }
  if (a.partials == nullptr) return;
  __syncthreads();
  // in whole lines: a column's place in the vectors is its own + lead, which all rows of a CTA share
  const float* sums = reinterpret_cast<const float*>(s_acc);
  float* part = a.partials + (int64_t)blockIdx.x * 2 * a.cols;
  for (int i = threadIdx.x; i < 2 * a.cols; i += 1024) {
    const int which = i >= a.cols, place = i - which * a.cols + c.lead;
    const int quad = which * kQuads + place % kVec / 4;
    part[i] = sums[(quad * n_vecs + place / kVec) * 4 + place % 4];
  }
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
  if (c < 2 * cols) {
#pragma unroll 8
    for (int i = slice; i < parts; i += 8) t += partials[(int64_t)i * 2 * cols + c];
  }
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

// Persistent grid of one CTA per SM, no more than there are rows for; a multiple of 8 where rows start
// inside vectors (see lead above).
int grid_of(int64_t rows, int groups, bool aligned) {
  const int64_t ctas = (rows + groups - 1) / groups;
  const int most = num_sms();
  if (aligned) return (int)(ctas < most ? ctas : most);
  return (int)(ctas < most / 8 * 8 ? (ctas + 7) / 8 * 8 : most / 8 * 8);
}

// With at most this many rows each gets its own CTA, and the parameters are read straight from
// memory: several groups a CTA would leave SMs idle and pay for staging the parameters.
constexpr int kFewRows = 2 * 148;

template <typename Kernel>
cudaError_t launch_norm(Kernel kernel, int grid, int threads, size_t smem, const NormArgs& a, cudaStream_t stream) {
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(grid), dim3(threads), smem, stream, a);
}

int vec_of(int dtype) { return dtype == NVFP4MOE_FP32 ? 4 : 8; }
// Columns that a row may span counted from an aligned vector's start.
int span_of(int cols, int vec) { return cols % vec == 0 ? cols : cols + vec - 1; }

// Shapes by row width, the first that holds the row (BF16, 16384 x 3060: 52 us forward and 78 backward on 96 threads, 76
// and 84 on 128): threads of a group x elements a thread, and groups per CTA, 512 threads an SM
// (forward works on two 16-bit rows at a time, backward holds the column sums: both about 128
// registers).  FP32 rows, twice the bytes for the same instructions, go one at a time, and backward takes
// half the groups, so that the rings stay deep.
template <int kType, bool kAligned, int kG, int kPer, int kGroups, int kParams>
cudaError_t forward_go(const NormArgs& a, cudaStream_t stream) {
  if (a.rows <= kFewRows)
    return launch_norm(norm_forward_kernel<kType, kAligned, kG, kPer, 1, 1, 0>, grid_of(a.rows, 1, kAligned), kG,
                       Ring<kType, kAligned, kG, kPer, 1, 1, 0>::kBytes, a, stream);
  // wide rows that start inside vectors: the parameters shifted in shared memory, and one row at a time
  constexpr int kR = kType == NVFP4MOE_FP32 || kG > 512 || (kG == 512 && !kAligned) ? 1 : 2;
  // FP32: twice the threads with half the elements each, 768 an SM (8192 x 5120: 64.5 -> 56 us)
  constexpr int kFold = kType == NVFP4MOE_FP32 && kPer == 32 && kG <= 256 ? 2 : 1;
  constexpr int kThreads = kG * kFold, kElems = kPer / kFold;
  constexpr int kTeams = kFold == 1 ? kGroups : 768 / kThreads > 1 ? 768 / kThreads : 1;
  return launch_norm(norm_forward_kernel<kType, kAligned, kThreads, kElems, kTeams, kR, kParams>,
                     grid_of(a.rows, kTeams, kAligned), kThreads * kTeams,
                     Ring<kType, kAligned, kThreads, kElems, kTeams, kR, kParams>::kBytes, a, stream);
}

template <int kType, bool kAligned>
cudaError_t forward_ring(const NormArgs& a, cudaStream_t stream) {
  const int span = span_of(a.cols, vec_of(kType));
  if (span <= 256) return forward_go<kType, kAligned, 32, 8, 16, 2>(a, stream);
  if (span <= 1024) return forward_go<kType, kAligned, 32, 32, 16, 2>(a, stream);
  if (span <= 2048) return forward_go<kType, kAligned, 64, 32, 8, 2>(a, stream);
  if (span <= 96 * 32) return forward_go<kType, kAligned, 96, 32, 5, 2>(a, stream);
  if (span <= 4096) return forward_go<kType, kAligned, 128, 32, 4, 2>(a, stream);
  if (span <= 5120) return forward_go<kType, kAligned, 160, 32, 3, 2>(a, stream);
  if (span <= 6144) return forward_go<kType, kAligned, 192, 32, 2, 2>(a, stream);
  if (span <= 8192) return forward_go<kType, kAligned, 256, 32, 2, 2>(a, stream);
  if (span <= 16384) return forward_go<kType, kAligned, 512, 32, 1, kAligned ? 0 : 2>(a, stream);
  return forward_go<kType, kAligned, 928, 32, 1, 0>(a, stream);
}

// Backward: the widest row of the ring kernel, and its groups.
constexpr int kBackwardWidest = 16384;
constexpr int backward_groups(int g16, bool f32) { return f32 ? (g16 + 1) / 2 : g16; }
int backward_groups_of(int span, bool f32, bool aligned) {
  const int g16 = span <= 1024 ? 16 : span <= 2048 ? 8 : span <= 96 * 32 ? 5 : span <= 4096 ? 4
                  : span <= 5120 ? (f32 || !aligned ? 3 : 2) : span <= 8192 ? 2 : 1;
  return backward_groups(g16, f32);
}

template <int kType, bool kAligned, int kG, int kPer, int kGroups16>
cudaError_t backward_go(const NormArgs& a, int ctas, cudaStream_t stream) {
  constexpr int kGroups = backward_groups(kGroups16, kType == NVFP4MOE_FP32);
  if (a.rows <= kFewRows)
    return launch_norm(norm_backward_kernel<kType, kAligned, kG, kPer, 1, 0>, ctas, kG,
                       Ring<kType, kAligned, kG, kPer, 1, 2, 0>::kBytes, a, stream);
  return launch_norm(norm_backward_kernel<kType, kAligned, kG, kPer, kGroups, 1>, ctas, kG * kGroups,
                     Ring<kType, kAligned, kG, kPer, kGroups, 2, 1>::kBytes, a, stream);
}

template <int kType, bool kAligned>
cudaError_t backward_ring(const NormArgs& a, int ctas, cudaStream_t stream) {
  const int span = span_of(a.cols, vec_of(kType));
  if (span <= 256) return backward_go<kType, kAligned, 32, 8, 16>(a, ctas, stream);
  if (span <= 1024) return backward_go<kType, kAligned, 32, 32, 16>(a, ctas, stream);
  if (span <= 2048) return backward_go<kType, kAligned, 64, 32, 8>(a, ctas, stream);
  if (span <= 96 * 32) return backward_go<kType, kAligned, 96, 32, 5>(a, ctas, stream);
  if (span <= 4096) return backward_go<kType, kAligned, 128, 32, 4>(a, ctas, stream);
  if (span <= 5120) {
    // 16-bit whole vectors: 320 threads x 16 elements against 160 x 32 for 32768 rows of 4104, 4608 and 5120 columns: 184,
    // 191 and 198 us against 188, 198 and 216; 1000 rows 16.0 to 17.1 against 17.6 to 18.6; 200 rows 7.7 to 9.0
    // against 9.1 to 9.7.  FP32 and rows that start inside vectors: slower
    if constexpr (kType != NVFP4MOE_FP32 && kAligned) return backward_go<kType, kAligned, 320, 16, 2>(a, ctas, stream);
    else return backward_go<kType, kAligned, 160, 32, 3>(a, ctas, stream);
  }
  if (span <= 6144) return backward_go<kType, kAligned, 192, 32, 2>(a, ctas, stream);
  if (span <= 8192) return backward_go<kType, kAligned, 256, 32, 2>(a, ctas, stream);
  return backward_go<kType, kAligned, 512, 32, 1>(a, ctas, stream);
}

int backward_ctas(int64_t rows, int cols, int vec) {
  const int span = span_of(cols, vec);
  const int groups = span > kBackwardWidest || rows <= kFewRows ? 1 : backward_groups_of(span, vec == 4, cols % vec == 0);
  return grid_of(rows, groups, cols % vec == 0);
}

template <int kType, bool kAligned>
cudaError_t backward_wide(const NormArgs& a, int ctas, cudaStream_t stream) {
  const int n_vecs = (span_of(a.cols, vec_of(kType)) + vec_of(kType) - 1) / vec_of(kType);
  const size_t smem = (size_t)n_vecs * vec_of(kType) * 2 * sizeof(float);
  const auto kernel = norm_backward_wide_kernel<kType, kAligned>;
  // the limit for the widest row, whatever this call's: see allow_smem
  constexpr size_t kWidest = (size_t)(kNormMaxCols + 8) * 2 * sizeof(float);
  static_assert(kWidest + 1024 <= 232448, "shared memory exceeds the per-block limit");
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), kWidest);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(ctas), dim3(1024), smem, stream, a, n_vecs);
}

template <int kType>
cudaError_t forward_type(const NormArgs& a, cudaStream_t stream) {
  return a.cols % vec_of(kType) == 0 ? forward_ring<kType, true>(a, stream) : forward_ring<kType, false>(a, stream);
}

template <int kType>
cudaError_t backward_type(const NormArgs& a, int ctas, cudaStream_t stream) {
  const bool aligned = a.cols % vec_of(kType) == 0;
  if (span_of(a.cols, vec_of(kType)) > kBackwardWidest)
    return aligned ? backward_wide<kType, true>(a, ctas, stream) : backward_wide<kType, false>(a, ctas, stream);
  return aligned ? backward_ring<kType, true>(a, ctas, stream) : backward_ring<kType, false>(a, ctas, stream);
}

}  // namespace

// As many as grid_of can give for up to `rows` rows of any width and type: few rows take a CTA each, more rows
// share CTAs, so the grid of more rows may be the smaller one.
int norm_backward_parts(int64_t rows) {
  const int most = num_sms();
  return (int)(rows < most ? (rows + 7) / 8 * 8 < most ? (rows + 7) / 8 * 8 : most : most);
}

cudaError_t launch_norm_forward(const NormArgs& a, int32_t* launches, cudaStream_t stream) {
  cudaError_t e;
  switch (a.dtype) {
    case NVFP4MOE_BF16: e = forward_type<NVFP4MOE_BF16>(a, stream); break;
    case NVFP4MOE_FP16: e = forward_type<NVFP4MOE_FP16>(a, stream); break;
    default: e = forward_type<NVFP4MOE_FP32>(a, stream);
  }
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_norm_backward(const NormArgs& a, int32_t* launches, cudaStream_t stream) {
  const int ctas = backward_ctas(a.rows, a.cols, vec_of(a.dtype));
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
