// Internal launchers of the FP8 (E4M3, 128-wide scale blocks) kernels.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace nvfp4 {

constexpr int kFp8Block = 128;             // K elements (and weight rows) under one scale
constexpr int kFp8MaxExperts = 1024;
constexpr uint32_t kFp8SkipFirstStage = 1u;   // = kDebugSkipFirstStage (kernels.h)

struct Fp8QuantArgs {
  const void* x;                   // [rows, cols] (silu: [rows, 2 * cols], gate then up)
  int64_t rows, cols, ld;
  const int32_t* route_pos;        // [rows, fanout] positions of each row's copies; NULL: row i -> i
  int32_t fanout;
  int32_t silu;
  uint8_t* codes;                  // [out_rows, cols], row stride ldq
  int64_t ldq;
  float* scales;                   // [ceil(cols / 128), out_rows]
  int64_t out_rows;
  int* status;
};

cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_fp8_quantize_weights(const void* w, int32_t E, int64_t N, int64_t K,
                                        uint8_t* codes, float* scales, int dtype, cudaStream_t s);

// fp8_rows.cu: quantisation and product of few rows in one launch, on the CUDA
// cores: up to kFp8FewRows rows of one matrix, or kFp8FewRoutes routes.
constexpr int kFp8FewRows = 4;
constexpr int kFp8FewRoutes = 16;
struct Fp8RowsArgs {
  const void* x;                   // [T, K] (silu: [T, 2 K]), row stride ld
  int64_t ld;
  int32_t silu;
  const int32_t* route_pos;        // grouped: [n_pos], or NULL
  int32_t n_pos, fanout;
  const uint8_t* w;
  const float* sw;                 // [E, nnb, nkb]
  const int32_t* offsets;          // grouped: [E + 1]; NULL: one matrix
  int32_t E;
  int32_t R;                       // rows of the output
  int32_t N, K, nkb, nnb;
  void* out;                       // [R, ldc], type of x
  int64_t ldc;
  int* status;
};
cudaError_t init_fp8_rows_attributes();
bool fp8_few_rows(int64_t R, int64_t n_pos, int64_t N, int64_t K, bool grouped);
cudaError_t launch_fp8_rows(const Fp8RowsArgs& a, int dtype, int sms, cudaStream_t s);

struct Fp8GemmArgs {
  const float* sa;                 // [nkb, lds]: scale of row m's K block b at b * lds + m
  int64_t lds;
  const float* sw;                 // [E, nnb, nkb]
  const int32_t* offsets;          // grouped: [E + 1]; NULL: one matrix
  int32_t E;
  int32_t rows;                    // M, or R
  int32_t N, K;
  int32_t nkb, nnb;                // 128-wide blocks of K and N
  void* out;                       // [rows, ldc]
  int64_t ldc;
  int32_t out_type;                // nvfp4_dtype
  int32_t vec;                     // every row of out is 16-byte aligned
  int32_t overlap;                 // start while the kernel before (the quantiser) still runs
  int* status;
  uint64_t timeout_ns;
  uint32_t debug_flags;
};

// fp8_gemm.cu.  ta: codes of the activations (boxes of fp8_tile_tokens() rows x
// 128 bytes), tw: of the weights ([E, N, K], boxes of 128 x 128).
cudaError_t init_fp8_gemm_attributes();
// Tokens per tile (16, 32, 64 or 128) of a product over `rows` rows; E = 0: one
// matrix.
int fp8_tile_tokens(int64_t rows, int32_t E);
cudaError_t launch_fp8_gemm(const CUtensorMap& ta, const CUtensorMap& tw, const Fp8GemmArgs& a,
                            int sms, cudaStream_t s);

}  // namespace nvfp4
