// FP8 block-scaled product of few rows, quantisation included, in one launch:
//
//   y[m, n] = sum_k (sa[m, k / 128] qa[m, k]) * sw[n / 128, k / 128] qw[n, k]
//
// For one to four rows the weights' bytes are all there is to move and the fixed
// cost of the tensor-core path (a quantiser launch, tensor memory, the sum over a
// cluster) is longer than moving them.  Here every block quantises the rows for
// itself (the same codes as the quantiser's; K values, read from L2) and keeps
// the codes' values in shared memory as FP32, their scales beside them; each warp
// then streams two weight rows, 16 bytes a lane and row, four steps on their way
// ahead, expands the codes exactly (E4M3 -> FP16 -> FP32) and adds 16 products in
// FP32 before both scales, multiplied first, are applied: the sum of code products
// stays below 16 * 448^2 and sa * sw in the range of the result, so that a row
// near the type's largest values comes out as on the tensor cores.  With fewer
// weight rows than warps the warps of a block share the rows' K.
//
// Grouped: one block column per route (blockIdx.y): the route's expert and, with
// route_pos, its token are found by the block's threads side by side.
// Bound: the weights' bytes (HBM or L2).
#include "fp8.h"
#include "fp8_quant.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 2;             // weight rows a warp streams
constexpr int kSteps = 4;            // steps of 512 K on their way

// Output of the block's rows: type by row format.
template <int DT>
__device__ __forceinline__ void put(void* out, int64_t at, float v) {
  static_cast<uint16_t*>(out)[at] = static_cast<uint16_t>(f32_to_elem<DT>(v));
}

template <int DT, int M, bool GROUPED, bool SILU>
__global__ void __launch_bounds__(kThreads) fp8_rows_kernel(const Fp8RowsArgs a, int ks) {
  // code values [M][steps][4][32] (conflict-free 16-byte reads), scales [M][steps][4]
  extern __shared__ float4 xs[];
  __shared__ float part[kWarps][kRows][M];
  __shared__ int route[2];           // expert, token
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int steps = (a.K + 511) / 512;
  float* xscale = reinterpret_cast<float*>(xs + M * steps * 128);
  const int per_block = kRows * (kWarps / ks);         // weight rows
  const int n0 = blockIdx.x * per_block + kRows * (warp / ks);
  const int kpart = warp % ks;
  int64_t row0 = 0;
  int e = 0;
  if constexpr (GROUPED) {
    const int r = blockIdx.y;
    if (threadIdx.x < 2) route[threadIdx.x] = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.E; i += kThreads) {
      const int lo = __ldg(a.offsets + i), hi = __ldg(a.offsets + i + 1);
      if (lo < 0 || hi < lo || hi > a.R) raise_status(a.status, NVFP4_ERR_DEVICE_CHECK);
      else if (lo <= r && r < hi) route[0] = i;
    }
    if (a.route_pos) {
      for (int i = threadIdx.x; i < a.n_pos; i += kThreads) {
        const int p = __ldg(a.route_pos + i);
        if (p >= a.R) raise_status(a.status, NVFP4_ERR_DEVICE_CHECK);
        else if (p == r) route[1] = i / a.fanout;
      }
    } else if (threadIdx.x == 0) {
      route[1] = r;
    }
    __syncthreads();
    e = route[0];
    row0 = route[1];
    if (e < 0 || row0 < 0) {                            // a row of no route
      const int n = blockIdx.x * per_block + static_cast<int>(threadIdx.x);
      if (static_cast<int>(threadIdx.x) < per_block && n < a.N)
        put<DT>(a.out, static_cast<int64_t>(r) * a.ldc + n, 0.f);
      return;
    }
  }
  const uint8_t* w[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    w[i] = a.w + (static_cast<int64_t>(e) * a.N + min(n0 + i, a.N - 1)) * a.K;
  const float* sw = a.sw + (static_cast<int64_t>(e) * a.nnb + min(n0, a.N - 1) / kFp8Block) * a.nkb;

  struct Batch {
    uint4 q[kSteps][kRows];
    float s[kSteps];
  };
  auto fetch = [&](Batch& b, int s0) {
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int k = (s0 + u * ks) * 512 + lane * 16;
      const bool in = k < a.K;                          // K % 16 == 0
      b.s[u] = in ? __ldg(sw + k / kFp8Block) : 0.f;
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        b.q[u][i] = in ? __ldg(reinterpret_cast<const uint4*>(w[i] + k)) : make_uint4(0, 0, 0, 0);
    }
  };
  Batch cur, next;
  fetch(cur, kpart);                                    // on their way while x is quantised

#pragma unroll
  for (int m = 0; m < M; ++m) {
    for (int s = warp; s < steps; s += kWarps) {
      const int k = s * 512 + lane * 16;
      float v[16];
      if (k < a.K) {
        load_row16<DT, SILU>(a.x, (row0 + m) * a.ld, a.K, k, v);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.f;
      }
      const BlockScale b(block_amax(v));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        xs[((m * steps + s) * 4 + j) * 32 + lane] =
            e4m3x4_f32(e4m3x4(b.quotient(v[4 * j]), b.quotient(v[4 * j + 1]),
                              b.quotient(v[4 * j + 2]), b.quotient(v[4 * j + 3])));
      if ((lane & 7) == 0) xscale[(m * steps + s) * 4 + (lane >> 3)] = b.scale;
    }
  }
  __syncthreads();

  float acc[kRows][M];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int m = 0; m < M; ++m) acc[i][m] = 0.f;
  for (int s0 = kpart; s0 < steps; s0 += kSteps * ks) {
    fetch(next, s0 + kSteps * ks);
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int s = s0 + u * ks;
      if (s >= steps) break;
      float sum[kRows][M];
#pragma unroll
      for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int m = 0; m < M; ++m) sum[i][m] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float4 q[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          q[i] = e4m3x4_f32(reinterpret_cast<const uint32_t*>(&cur.q[u][i])[j]);
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const float4 x = xs[((m * steps + s) * 4 + j) * 32 + lane];
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            sum[i][m] = fmaf(x.w, q[i].w, fmaf(x.z, q[i].z, fmaf(x.y, q[i].y,
                                                             fmaf(x.x, q[i].x, sum[i][m]))));
        }
      }
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const float f = xscale[(m * steps + s) * 4 + (lane >> 3)] * cur.s[u];
#pragma unroll
        for (int i = 0; i < kRows; ++i) acc[i][m] = fmaf(sum[i][m], f, acc[i][m]);
      }
    }
    cur = next;
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[i][m] += __shfl_xor_sync(0xFFFFFFFFu, acc[i][m], o);
      if (lane == 0) part[warp][i][m] = acc[i][m];
    }
  __syncthreads();
  // one thread per weight row and row of x: the K parts in order
  if (threadIdx.x < per_block * M) {
    const int i = threadIdx.x % per_block, m = threadIdx.x / per_block;
    const int first = i / kRows * ks;
    float v = 0.f;
    for (int j = 0; j < ks; ++j) v += part[first + j][i % kRows][m];
    const int n = blockIdx.x * per_block + i;
    const int64_t r = GROUPED ? static_cast<int64_t>(blockIdx.y) : m;
    if (n < a.N) put<DT>(a.out, r * a.ldc + n, v);
  }
}

constexpr size_t kMaxSmem = 160 * 1024;
constexpr int64_t kStepBytes = 512 * 4 + 4 * 4;      // 512 code values and four scales

template <int DT, int M, bool GROUPED, bool SILU>
cudaError_t go(const Fp8RowsArgs& a, int sms, cudaStream_t s) {
  // warps share the K of their rows while the blocks would not cover the SMs twice
  int ks = 1;
  const int64_t columns = GROUPED ? a.R : 1;
  while (ks < kWarps && (a.N * ks + kRows * kWarps - 1) / (kRows * kWarps) * columns < 2LL * sms &&
         (a.K + 511) / 512 >= 4 * ks)
    ks *= 2;
  const int per_block = kRows * (kWarps / ks);
  const size_t smem = static_cast<size_t>(M * ((a.K + 511) / 512) * kStepBytes);
  const dim3 grid(static_cast<unsigned>((a.N + per_block - 1) / per_block),
                  static_cast<unsigned>(columns), 1);
  fp8_rows_kernel<DT, M, GROUPED, SILU><<<grid, kThreads, smem, s>>>(a, ks);
  return cudaGetLastError();
}

template <int DT>
cudaError_t by_rows(const Fp8RowsArgs& a, int sms, cudaStream_t s) {
  if (a.offsets) return a.silu ? go<DT, 1, true, true>(a, sms, s) : go<DT, 1, true, false>(a, sms, s);
  switch (a.R) {
    case 1: return go<DT, 1, false, false>(a, sms, s);
    case 2: return go<DT, 2, false, false>(a, sms, s);
    case 3: return go<DT, 3, false, false>(a, sms, s);
    default: return go<DT, 4, false, false>(a, sms, s);
  }
}

template <int DT, int M, bool GROUPED, bool SILU>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(fp8_rows_kernel<DT, M, GROUPED, SILU>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kMaxSmem));
}

template <int DT>
cudaError_t set_all() {
  cudaError_t e = set_smem<DT, 1, true, true>();
  if (e == cudaSuccess) e = set_smem<DT, 1, true, false>();
  if (e == cudaSuccess) e = set_smem<DT, 1, false, false>();
  if (e == cudaSuccess) e = set_smem<DT, 2, false, false>();
  if (e == cudaSuccess) e = set_smem<DT, 3, false, false>();
  if (e == cudaSuccess) e = set_smem<DT, 4, false, false>();
  return e;
}

}  // namespace

cudaError_t init_fp8_rows_attributes() {
  const cudaError_t e = set_all<NVFP4_BF16>();
  return e == cudaSuccess ? set_all<NVFP4_FP16>() : e;
}

// Where this path is the faster one: it takes about 2.5 us + 0.13 + 0.14 M us per
// MB of weights (the codes' expansion and M additions a weight are what it
// spends), the tensor-core path about 6.2 us + 0.16 us per MB: one row of 4096 x
// 6144 9.2 us here and 9.7 us there, of 512 x 512 2.8 and 6.2 us, of 8192 x 8192
// 17.4 and 16.7 us; four rows of 4096 x 6144 20.1 and 9.9 us.  So M times the
// weights' bytes up to 32 MB.  Grouped, each route brings weights of its own, from
// HBM: 16 routes of 1024 x 2048 14.3 us here, 18 there 12.9 us, 8 here 8.1 us;
// up to 20 MB.
bool fp8_few_rows(int64_t R, int64_t n_pos, int64_t N, int64_t K, bool grouped) {
  if (R > (grouped ? kFp8FewRoutes : kFp8FewRows) || n_pos > 4 * kFp8FewRoutes) return false;
  if ((grouped ? 1 : R) * ((K + 511) / 512) * kStepBytes > static_cast<int64_t>(kMaxSmem)) return false;
  return R * N * K <= ((grouped ? 20LL : 32LL) << 20);
}

cudaError_t launch_fp8_rows(const Fp8RowsArgs& a, int dtype, int sms, cudaStream_t s) {
  return dtype == NVFP4_BF16 ? by_rows<NVFP4_BF16>(a, sms, s) : by_rows<NVFP4_FP16>(a, sms, s);
}

}  // namespace nvfp4
