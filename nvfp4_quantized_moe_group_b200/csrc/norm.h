// Interface of the layer norm kernels (norm.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace nvfp4moe {

constexpr int kNormMaxCols = 28672;   // two FP32 column sums of a row fit a CTA's shared memory

struct NormArgs {
  const void* x;         // [rows][cols]
  const float* gamma;    // [cols] or nullptr (ones)
  const float* beta;     // [cols] or nullptr (zeros); forward, layer form
  float* mean;           // [rows]; layer form (forward: out, may be nullptr)
  float* rstd;           // [rows] (forward: out, may be nullptr)
  void* y;               // forward: [rows][cols]
  const void* dy;        // backward
  void* dx;
  float* dgamma;         // [cols] or nullptr
  float* dbeta;          // [cols] or nullptr
  float* partials;       // norm_backward_parts() * 2 * cols floats, with dgamma or dbeta
  int64_t rows;
  int cols;
  float eps;
  int rms;
  int dtype;             // NVFP4MOE_BF16 / _FP16 / _FP32
};

// The most CTAs that the backward pass of up to `rows` rows takes: what the workspace is sized for.
int norm_backward_parts(int64_t rows);
cudaError_t launch_norm_forward(const NormArgs& a, int* launches, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormArgs& a, int* launches, cudaStream_t stream);

}  // namespace nvfp4moe
