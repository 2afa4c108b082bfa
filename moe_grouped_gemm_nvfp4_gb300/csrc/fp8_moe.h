// Internal launcher of the MoE layer for a few tokens (fp8_moe.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "gate.cuh"

namespace nvfp4 {

constexpr int kMoeMaxTokens = 16;
constexpr int kMoeMaxRoutes = 256;

struct Fp8MoeArgs {
  const void* x;                   // [T, K] BF16 or FP16, row stride ld
  int64_t ld;
  const void* router;              // [E, K] (dense), or NULL: ids and weights are given
  int32_t router_type;             // nvfp4_dtype
  GateRule rule;                   // E and topk always; the rest with a router
  int32_t T, K, I, N;
  const uint8_t* w1;               // codes [E, 2 I, K]: gate half, up half
  const float* s1;                 // [E, ceil(2 I / 128), ceil(K / 128)]
  const uint8_t* w2;               // codes [E, N, I]
  const float* s2;                 // [E, ceil(N / 128), ceil(I / 128)]
  int32_t* ids;                    // [T, topk]
  float* weights;                  // [T, topk]
  void* out;                       // [T, N], type of x, row stride ldo
  int64_t ldo;
  float* logits;                   // workspace [T, E]
  float* h;                        // workspace [T * topk, I]
  float* part;                     // workspace [T * topk, N]
  uint32_t* arrived;               // workspace [ceil(N / 16)]
  int* status;
};

struct Fp8MoePlan {
  int stages, tiles;               // ring stages of a warp; 8-token tiles
  int act_stride, act_rows;        // activations in shared memory
  size_t smem;
  int grid;
};
// Whether the sizes fit the kernel, and its shape.
bool fp8_moe_plan(int T, int topk, int E, int64_t K, int64_t I, int64_t N, int sms, Fp8MoePlan* p);
cudaError_t init_fp8_moe_attributes();
cudaError_t launch_fp8_moe(const Fp8MoeArgs& a, const Fp8MoePlan& p, int dtype, cudaStream_t s);

}  // namespace nvfp4
