// Element access of BF16, FP16 and FP32 rows: VEC elements in one access,
// held as floats.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "common.cuh"

namespace nvfp4 {

// DT: nvfp4_dtype
template <int DT> struct Elem { using Bits = uint16_t; };
template <> struct Elem<NVFP4_FP32> { using Bits = uint32_t; };
template <int DT> constexpr int elem_bytes() { return sizeof(typename Elem<DT>::Bits); }
template <int DT> constexpr int elems_per_16b() { return 16 / elem_bytes<DT>(); }

template <int DT>
__device__ __forceinline__ float elem_to_f32(uint32_t bits) {
  if constexpr (DT == NVFP4_BF16) return bf16_bits_to_f32(bits);
  else if constexpr (DT == NVFP4_FP16)
    return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
  else return __uint_as_float(bits);
}

template <int DT>
__device__ __forceinline__ uint32_t f32_to_elem(float f) {
  if constexpr (DT == NVFP4_BF16) return f32_to_bf16_rn(f);
  else if constexpr (DT == NVFP4_FP16) return __half_as_ushort(__float2half_rn(f));
  else return __float_as_uint(f);
}

// VEC elements as they lie in memory: one 16-byte word, or one element.
template <int DT, int VEC>
struct Pack {
  static constexpr int kWords = VEC * elem_bytes<DT>() >= 4 ? VEC * elem_bytes<DT>() / 4 : 1;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* base, int64_t elem) {
    using Bits = typename Elem<DT>::Bits;
    const Bits* p = static_cast<const Bits*>(base) + elem;
    if constexpr (VEC == 1) {
      w[0] = __ldg(p);
    } else {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (elem_bytes<DT>() == 4) return __uint_as_float(w[i]);
    else if constexpr (VEC == 1) return elem_to_f32<DT>(w[0]);
    else return elem_to_f32<DT>((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
  }
  __device__ __forceinline__ void from(const float (&f)[VEC]) {
    if constexpr (elem_bytes<DT>() == 4 || VEC == 1) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[i] = f32_to_elem<DT>(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i)
        w[i] = f32_to_elem<DT>(f[2 * i]) | (f32_to_elem<DT>(f[2 * i + 1]) << 16);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
};

}  // namespace nvfp4
