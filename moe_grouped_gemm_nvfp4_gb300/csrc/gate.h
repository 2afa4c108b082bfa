// Internal launchers of the top-k gate (gate.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gate.cuh"

namespace nvfp4 {

struct GateArgs {
  const void* logits;              // [T, E], row stride ld
  int64_t ld;
  int64_t T;
  GateRule rule;
  int32_t* ids;                    // [T, topk]
  float* weights;                  // [T, topk]
  const float* dweights;           // grad: [T, topk]
  const int32_t* chosen;           // grad: ids [T, topk]
  void* dlogits;                   // grad: dense [T, E], type of the logits
  int* status;
};

cudaError_t launch_topk_gate(const GateArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_topk_gate_grad(const GateArgs& a, int dtype, cudaStream_t s);

}  // namespace nvfp4
