// FP8 block quantisers.
//
// Activations, one scale per row and 128 columns: a = max |x| over the block
// (at least 2^-100), scale = a / 448, code = E4M3(448 x / a), rounded once from
// the real quotient (nearest, ties to even; fp8_quant.cuh).
//
// A lane holds 16 consecutive elements (two 16-byte loads, one 16-byte store),
// eight lanes a block, so the maximum needs three shuffles.  A row that goes to
// several route positions is read and rounded once and written to each.  Bound:
// HBM (2 bytes read + fanout * (1 + 4/128) written per element): 8192 x 8192 37 us,
// 8192 x 6144 to eight positions each 97 us, 0.8 of the copy rate; the scales,
// written four bytes at a time into their K-block-major matrix, are what it lacks.
#include <type_traits>

#include "fp8.h"
#include "fp8_quant.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

template <int DT, bool SILU>
__global__ void __launch_bounds__(kThreads) fp8_quantize_kernel(const Fp8QuantArgs a, int chunks) {
  // a GEMM launched to overlap this kernel may take its place on the SMs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = task / chunks;
  if (row >= a.rows) return;
  const int64_t c = (task - row * chunks) * 512 + lane * 16;
  const bool on = c < a.cols;                      // cols % 16 == 0: all 16 or none
  float v[16];
  if (on) {
    load_row16<DT, SILU>(a.x, row * a.ld, a.cols, c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
  }
  const float amax = block_amax(v);
  if (!on) return;
  const BlockScale b(amax);
  uint4 q;
  uint32_t* qw = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    qw[i] = e4m3x4(b.quotient(v[4 * i]), b.quotient(v[4 * i + 1]), b.quotient(v[4 * i + 2]),
                   b.quotient(v[4 * i + 3]));
  const int64_t kb = c / kFp8Block;
  const bool first = (c % kFp8Block) == 0;
  for (int k = 0; k < a.fanout; ++k) {
    int64_t r = row;
    if (a.route_pos) {
      r = __ldg(a.route_pos + row * a.fanout + k);
      if (r < 0) continue;
      if (r >= a.out_rows) { raise_status(a.status, NVFP4_ERR_DEVICE_CHECK); continue; }
    }
    *reinterpret_cast<uint4*>(a.codes + r * a.ldq + c) = q;
    if (first) a.scales[kb * a.out_rows + r] = b.scale;
  }
}

// Weights, one scale per 128 x 128 block (prepared once): a block of threads
// per weight block, the elements read twice.
template <int DT>
__global__ void __launch_bounds__(kThreads) fp8_quantize_weights_kernel(
    const void* w, int64_t N, int64_t K, int nnb, int nkb, uint8_t* codes, float* scales) {
  __shared__ float part[kThreads / 32];
  const int kb = blockIdx.x % nkb;
  const int64_t rest = blockIdx.x / nkb;
  const int nb = static_cast<int>(rest % nnb);
  const int64_t e = rest / nnb;
  const int64_t n0 = static_cast<int64_t>(nb) * kFp8Block, k0 = static_cast<int64_t>(kb) * kFp8Block;
  const int col = threadIdx.x & 127, half = threadIdx.x >> 7;
  const bool on = k0 + col < K;
  const int64_t base = (e * N + n0) * K + k0 + col;
  const int n_rows = static_cast<int>(N - n0 < kFp8Block ? N - n0 : kFp8Block);
  float amax = 0.f;
  if (on)
    for (int r = half; r < n_rows; r += 2) {
      Pack<DT, 1> v;
      v.load(w, base + r * K);
      amax = fmaxf(amax, fabsf(v.get(0)));
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) amax = fmaxf(amax, part[i]);
  const std::conditional_t<DT == NVFP4_FP32, BlockScale32, BlockScale> b(amax);
  if (on)
    for (int r = half; r < n_rows; r += 2) {
      Pack<DT, 1> v;
      v.load(w, base + r * K);
      codes[base + r * K] = static_cast<uint8_t>(e4m3x4(b.quotient(v.get(0)), 0.f, 0.f, 0.f));
    }
  if (threadIdx.x == 0) scales[(e * nnb + nb) * nkb + kb] = b.scale;
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, int dtype, cudaStream_t s) {
  const int chunks = static_cast<int>((a.cols + 511) / 512);
  const int64_t blocks = (a.rows * chunks + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  if (blocks == 0) return cudaSuccess;
  const unsigned g = static_cast<unsigned>(blocks);
  if (dtype == NVFP4_BF16) {
    if (a.silu) fp8_quantize_kernel<NVFP4_BF16, true><<<g, kThreads, 0, s>>>(a, chunks);
    else fp8_quantize_kernel<NVFP4_BF16, false><<<g, kThreads, 0, s>>>(a, chunks);
  } else {
    if (a.silu) fp8_quantize_kernel<NVFP4_FP16, true><<<g, kThreads, 0, s>>>(a, chunks);
    else fp8_quantize_kernel<NVFP4_FP16, false><<<g, kThreads, 0, s>>>(a, chunks);
  }
  return cudaGetLastError();
}

cudaError_t launch_fp8_quantize_weights(const void* w, int32_t E, int64_t N, int64_t K,
                                        uint8_t* codes, float* scales, int dtype,
                                        cudaStream_t s) {
  const int nnb = static_cast<int>((N + 127) / 128), nkb = static_cast<int>((K + 127) / 128);
  const int64_t blocks = static_cast<int64_t>(E) * nnb * nkb;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  if (blocks == 0) return cudaSuccess;
  const unsigned g = static_cast<unsigned>(blocks);
  if (dtype == NVFP4_BF16)
    fp8_quantize_weights_kernel<NVFP4_BF16><<<g, kThreads, 0, s>>>(w, N, K, nnb, nkb, codes, scales);
  else if (dtype == NVFP4_FP16)
    fp8_quantize_weights_kernel<NVFP4_FP16><<<g, kThreads, 0, s>>>(w, N, K, nnb, nkb, codes, scales);
  else
    fp8_quantize_weights_kernel<NVFP4_FP32><<<g, kThreads, 0, s>>>(w, N, K, nnb, nkb, codes, scales);
  return cudaGetLastError();
}

}  // namespace nvfp4
