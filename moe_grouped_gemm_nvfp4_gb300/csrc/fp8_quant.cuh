// E4M3 block quantisation, shared by the quantisers and the product for few
// rows (which quantises its rows itself, to the same codes and scales).
#pragma once

#include <cuda_fp16.h>

#include "rows.cuh"

namespace nvfp4 {
namespace {

constexpr float kAmaxFloor = 7.888609052210118e-31f;   // 2^-100

// Four floats -> four E4M3 codes, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Four E4M3 codes -> four floats, exactly.
__device__ __forceinline__ float4 e4m3x4_f32(uint32_t codes) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(codes));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(x.x, x.y, y.x, y.y);
}

// Scale of a block with largest magnitude amax, and the quotient 448 x / a of
// its elements: p = 0.875 x is exact for 16-bit x (448 = 0.875 * 2^9), q0 = p *
// (1 / a') with a' = a / 512 is within two ulp, and one residual step q0 + (p -
// q0 a') / a' (Markstein's FMA correction) returns a quotient that is
// representable exactly; an E4M3 rounding border has five significant bits, so it
// is met exactly or missed by at least 2^-16 of its value, far more than the
// step's error.  No overflow: p and a' stay below the largest float, q0 below
// 448 (1 + 2^-22).  That is quotient(); the gate's product, formed in FP32 with
// rounding errors of its own, takes it too.
struct BlockScale {
  float unit, inv, scale;
  __device__ __forceinline__ explicit BlockScale(float amax) {
    const float a = fmaxf(amax, kAmaxFloor);
    unit = a * 0.001953125f;
    inv = __frcp_rn(unit);
    scale = __fdiv_rn(a, 448.f);
  }
  __device__ __forceinline__ float quotient(float x) const {
    const float p = x * 0.875f;
    const float q = p * inv;
    return fmaf(fmaf(-q, unit, p), inv, q);
  }
};

// The quotient for FP32 x, where 0.875 x is a sum of two floats, p + pl, and may
// miss a border by 2^-29 of its value only.  The residual step with pl included
// returns the nearest float, which lies on the border or on the quotient's side of
// it; then the sign of what is left, (p - q a') + pl with the first term exact,
// moves a q of even mantissa (a border's is) one step towards the quotient.  Blocks
// below 2^-40 are scaled up (exactly) so that the residuals do not underflow.
// (Without all that one normal weight in two million got the neighbouring code.)
struct BlockScale32 {
  float up, unit, inv, scale;
  __device__ __forceinline__ explicit BlockScale32(float amax) {
    const BlockScale b(amax);
    const bool low = b.unit < 1.7763568394002505e-15f;     // 2^-49
    up = low ? 1.152921504606847e18f : 1.f;                // 2^60
    unit = b.unit * up;
    inv = low ? __frcp_rn(unit) : b.inv;
    scale = b.scale;
  }
  __device__ __forceinline__ float quotient(float x) const {
    const float xu = x * up;
    const float p = xu * 0.875f;
    const float pl = fmaf(xu, 0.875f, -p);
    float q = p * inv;
    q = fmaf(fmaf(-q, unit, p) + pl, inv, q);
    const float left = fmaf(-q, unit, p) + pl;
    const uint32_t bits = __float_as_uint(q);
    const bool away = ((bits ^ __float_as_uint(left)) >> 31) == 0;   // from zero
    return left != 0.f && (bits & 1u) == 0 ? __uint_as_float(bits + (away ? 1u : ~0u)) : q;
  }
};

// 16 elements of a row at column c, as floats; SILU: SiLU(row[c]) * row[cols + c].
template <int DT, bool SILU>
__device__ __forceinline__ void load_row16(const void* x, int64_t row_elem, int64_t cols, int64_t c,
                                           float (&v)[16]) {
  Pack<DT, 8> lo, hi;
  lo.load(x, row_elem + c);
  hi.load(x, row_elem + c + 8);
#pragma unroll
  for (int i = 0; i < 8; ++i) { v[i] = lo.get(i); v[8 + i] = hi.get(i); }
  if constexpr (SILU) {
    lo.load(x, row_elem + cols + c);
    hi.load(x, row_elem + cols + c + 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = v[i] / (1.f + __expf(-v[i])) * lo.get(i);
      v[8 + i] = v[8 + i] / (1.f + __expf(-v[8 + i])) * hi.get(i);
    }
  }
}

// Largest magnitude over the 8 lanes (of 16 elements each) of a block.
__device__ __forceinline__ float block_amax(const float (&v)[16]) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  return amax;
}

}  // namespace
}  // namespace nvfp4
