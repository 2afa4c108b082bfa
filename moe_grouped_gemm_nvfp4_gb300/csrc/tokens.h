// Internal launchers of the token movement kernels (tokens.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace nvfp4 {

struct TokensArgs {
  const void* src;                 // dispatch: x [T, D]; combine: y [R, D]; grad: dout [T, D]
  int64_t ld;                      // row stride of src, elements
  const void* y;                   // grad: y [R, D]
  int64_t ld_y;
  const int32_t* pos;              // [T, topk], -1: no route
  const float* w;                  // [T, topk]; combine: NULL = ones
  const int32_t* live;             // rows [*live, R) of the output are zeroed; NULL: none
  void* out;                       // dispatch: [R, D]; combine: [T, D]; grad: dy [R, D]
  float* dw;                       // grad: [T, topk]
  int64_t T, R;
  int32_t D;
  int32_t topk;
  int* status;
};

// dtype: nvfp4_dtype.  The launchers return cudaErrorInvalidConfiguration for
// a grid that does not fit (more than 2^31 - 1 blocks).
cudaError_t launch_tokens_dispatch(const TokensArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_tokens_combine(const TokensArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_tokens_combine_grad(const TokensArgs& a, int dtype, cudaStream_t s);

}  // namespace nvfp4
