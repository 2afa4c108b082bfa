// Internal launchers of the root-mean-square norm (norm.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace nvfp4 {

constexpr int kNormMaxWidth = 16384;       // 512 threads of 32 elements

struct NormArgs {
  const void* x;                   // [T, D], row stride ld (grad: h)
  int64_t ld;
  const void* r;                   // residual [T, D], row stride ld_r, or NULL (grad: dh)
  int64_t ld_r;
  const void* dy;                  // grad: [T, D], row stride ld_dy
  int64_t ld_dy;
  const void* w;                   // [D]
  int32_t w_type;                  // nvfp4_dtype
  int32_t D;
  int64_t T;
  float eps;
  void* h;                         // x + r, dense [T, D] (with a residual)
  void* y;                         // dense [T, D] (grad: dx)
  uint8_t* codes;                  // E4M3, dense [T, D]
  float* scales;                   // [ceil(D / 128), T]
  float* part;                     // grad: [parts, D]
  void* dw;                        // grad: [D], type of w
};

// Partial sums of the weight's gradient.
int norm_grad_parts(int64_t T, int64_t D, int dtype);
cudaError_t init_norm_attributes();
cudaError_t launch_rms_norm(const NormArgs& a, int dtype, bool fp8, cudaStream_t s);
cudaError_t launch_rms_norm_grad(const NormArgs& a, int dtype, cudaStream_t s);

}  // namespace nvfp4
