// Device helpers shared by the FP8 GEMM kernels: the kind::f8f6f4 MMA, 3-D TMA
// loads of the weights, packed FP32 accumulation and the map from work units
// to (expert, weight rows, tokens).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "fp8.h"

namespace nvfp4 {
namespace {

// Instruction descriptor of kind::f8f6f4: E4M3 x E4M3, FP32 accumulator,
// K-major A and B, M = m, N = n.
__device__ __forceinline__ uint32_t idesc_e4m3(uint32_t m, uint32_t n) {
  return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// D[tmem] (+)= A[smem] . B[smem]^T, K = 32, issued by one lane of a converged
// warp.
__device__ __forceinline__ void tc_mma_e4m3_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                  uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .pred e;\n\t.reg .b32 l;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync l|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void tma_load_3d_elect(uint32_t dst, const void* tmap, uint32_t bar,
                                                  int32_t x, int32_t y, int32_t z,
                                                  uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 l;\n\t"
      "elect.sync l|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;\n\t}"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z),
         "l"(policy)
      : "memory");
}

// acc += t * f on a pair of FP32 values (one instruction).
__device__ __forceinline__ void fma_pair(float& a0, float& a1, uint32_t t0, uint32_t t1, float f0,
                                         float f1) {
  asm("{\n\t.reg .b64 a, t, f;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 t, {%2, %3};\n\tmov.b64 f, {%4, %5};\n\t"
      "fma.rn.f32x2 a, t, f, a;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1) : "r"(t0), "r"(t1), "f"(f0), "f"(f1));
}

// One FP32 value as the output type's bits (16-bit types in the low half).
__device__ __forceinline__ uint16_t f32_to_out16(float f, int type) {
  return type == NVFP4_FP16 ? __half_as_ushort(__float2half_rn(f)) : f32_to_bf16_rn(f);
}

// Waits for a phase regardless of the abort flag, bounded by the timeout
// (draining copies and MMAs already in flight).
__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity, uint64_t timeout) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1; i < 0x7FFFFFFFu; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 31u) == 0 && globaltimer() - t0 > timeout) return false;
  }
  return false;
}

// Work units in the order expert, weight tile, token tile (token tiles of one
// weight tile are neighbours, so the second one finds the weights in L2).
struct UnitMap {
  const int* first;        // grouped: row offsets [E + 1] (shared memory); NULL: one matrix
  const int* tiles;        // grouped: token tiles of the experts before e [E + 1]
  int E, rows, ntiles, ttiles, width;
};
struct Unit {
  int e, nt, row, cnt;     // expert, weight tile, first token row, rows of the tile
};

__device__ __forceinline__ int unit_count(const UnitMap& m) {
  return (m.first ? m.tiles[m.E] : m.ttiles) * m.ntiles;
}

__device__ __forceinline__ Unit unit_at(const UnitMap& m, int u) {
  Unit r;
  if (!m.first) {
    r.e = 0;
    r.nt = u / m.ttiles;
    const int t = u - r.nt * m.ttiles;
    r.row = t * m.width;
    r.cnt = min(m.width, m.rows - r.row);
    return r;
  }
  const int q = u / m.ntiles;
  int lo = 0, hi = m.E;                       // tiles[lo] <= q < tiles[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (m.tiles[mid] <= q) lo = mid; else hi = mid;
  }
  const int tc = m.tiles[lo + 1] - m.tiles[lo];
  const int local = u - m.tiles[lo] * m.ntiles;
  r.e = lo;
  r.nt = local / tc;
  const int t = local - r.nt * tc;
  r.row = m.first[lo] + t * m.width;
  r.cnt = min(m.width, m.first[lo + 1] - r.row);
  return r;
}

// Fills first/tiles from the device offsets (whole block; one warp scans).
// An expert whose offsets are not monotone inside [0, rows] counts as empty
// and the error is recorded.
__device__ __forceinline__ void load_units(const int32_t* offsets, int E, int rows, int width,
                                           int* first, int* tiles, int* status) {
  for (int i = threadIdx.x; i <= E; i += blockDim.x) first[i] = __ldg(offsets + i);
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      int n = 0;
      if (e < E) {
        const int a = first[e], b = first[e + 1];
        if (a < 0 || b < a || b > rows) raise_status(status, NVFP4_ERR_DEVICE_CHECK);
        else n = (b - a + width - 1) / width;
      }
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
      }
      if (e < E) tiles[e] = base + incl - n;
      base += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (lane == 0) tiles[E] = base;
  }
  __syncthreads();
}

// Zeros the output rows from `first` on (routes that no expert took); one
// warp of each block, the blocks taking rows in turn.
__device__ __forceinline__ void zero_rows_past(const Fp8GemmArgs& a, int first, int lane) {
  const int es = a.out_type == NVFP4_FP32 ? 4 : 2;
  for (int64_t r = max(first, 0) + static_cast<int>(blockIdx.x); r < a.rows; r += gridDim.x) {
    uint16_t* row = static_cast<uint16_t*>(a.out) + r * a.ldc * (es / 2);
    for (int i = lane; i < a.N * (es / 2); i += 32) row[i] = 0;
  }
}

}  // namespace
}  // namespace nvfp4
