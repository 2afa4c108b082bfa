// Internal launcher of the MoE layer for a few tokens (fp8_moe.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "gate.cuh"

namespace nvfp4 {

// More tokens go through launches for any number (router product, gate, layout, two products,
// sum).  In graphs, 128 experts, this call and those: 8 of 128 of 6144 x 2048, one token 61
// and 73 us, 2 tokens 108 and 114, 4 tokens 178 and 179, 8 tokens 305 and 300; of 2048 x 768 26
// and 39, 33 and 41, 47 and 51, 61 and 65 us; 2 of 128 of 1040 x 528 21 and 19 us, 25 and 20, 26
// and 27, 28 and 40.  Without a graph the host's time comes to those, several calls; this is one
// of 9 us.  And those round gate_up's product and the experts' rows to 16 bits.
constexpr int kMoeMaxTokens = 8;
constexpr int kMoeMaxRoutes = 256;           // one thread each
constexpr int kMoeMaxGrid = 160;

struct Fp8MoeArgs {
  const void* x;                   // [T, K] BF16 or FP16, row stride ld
  int64_t ld;
  int32_t type;                    // nvfp4_dtype of x and out
  const void* router;              // [E, K] (dense), or NULL: ids and weights are given
  int32_t router_type;             // nvfp4_dtype
  GateRule rule;                   // E and topk always; the rest with a router
  int32_t T, K, I, N;
  const float* s1;                 // gate_up scales [E, ceil(2 I / 128), ceil(K / 128)]
  const float* s2;                 // down scales [E, ceil(N / 128), ceil(I / 128)]
  int32_t* ids;                    // [T, topk]
  float* weights;                  // [T, topk]
  void* out;                       // [T, N], type of x, row stride ldo
  int64_t ldo;
  // workspace (MoeLayout)
  float* logits;                   // [T, E]
  uint8_t* xq;                     // codes of x [columns, ld_xq]
  int64_t ld_xq;
  float* xs;                       // scales [blocks of K][columns]
  uint8_t* hq;                     // codes of h [(experts + 1) * columns, ld_hq]
  int64_t ld_hq;
  float* hs;                       // scales [experts + 1][blocks of I][columns]
  float* part;                     // [2 * grid][2][columns][128]
  // runs of gate_up and of down that are taken, gate_up runs that are done, unused; then
  // what arrived of each of gate_up's items (items1) and four of each of down's
  uint32_t* counters;
  int32_t items1;                  // items of gate_up at most
  int32_t experts;                 // live ones at most
  int* status;
  uint64_t timeout_ns;
};

// Sizes that follow from a call's: token columns, live experts at most, and where the
// workspace's parts begin.
struct MoeLayout {
  int columns, experts;
  int64_t ld_xq, ld_hq;
  size_t xq, xs, hq, hs, part, counters, bytes;
};
// False for sizes that the kernel does not take.
bool fp8_moe_layout(int64_t T, int32_t topk, int32_t E, int64_t K, int64_t I, int64_t N,
                    MoeLayout* m);

cudaError_t init_fp8_moe_attributes();
// Rows of the maps' boxes of activations.
int fp8_moe_box_rows();
// t1: gate_up [2 E, I, K], t2: down [E, N, I] (boxes of 128 x 128); tx, th: codes of x
// and h (boxes of fp8_moe_box_rows() x 128).
cudaError_t launch_fp8_moe(const CUtensorMap& t1, const CUtensorMap& t2, const CUtensorMap& tx,
                           const CUtensorMap& th, const Fp8MoeArgs& a, int sms, cudaStream_t s);

}  // namespace nvfp4
