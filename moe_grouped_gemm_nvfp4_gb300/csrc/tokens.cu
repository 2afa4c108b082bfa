// Token rows into expert order and back ("The FP4 Frontier", Finding 5: the
// grouped GEMM wants each expert's token rows contiguous), in BF16, FP16 or
// FP32, and the gradients of both:
//
//   dispatch       out[pos[t,k]] = x[t]
//   combine        out[t] = sum_k w[t,k] y[pos[t,k]]   (w = 1: dispatch's gradient)
//   combine grad   dy[pos[t,k]] = w[t,k] dout[t],  dw[t,k] = <dout[t], y[pos[t,k]]>
//
// All three walk the tokens, not the routes: one token's row is read once (or
// written once) and its topk route rows are whole rows elsewhere, so every
// byte moves once and no sum needs an atomic -- the order of each sum is fixed
// (k ascending; columns by thread, lanes, warps) and results repeat bit for
// bit.  Sums are FP32, rounded once at the store.  Bound: HBM.
#include "rows.cuh"
#include "tokens.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kRoutes = 8;           // routes in flight per thread
constexpr int kTailBlocks = 152;     // blocks that zero the rows past the live ones

// A block covers `rows` tokens x `cols` column groups of VEC elements
// (rows * cols = 256 threads); narrow rows share a block.
struct Shape {
  int cols, rows;
  int64_t row_blocks, col_blocks;
};

Shape shape_of(int64_t T, int64_t groups, bool whole_rows) {
  Shape s;
  s.cols = 32;
  while (s.cols < kThreads && s.cols < groups) s.cols *= 2;
  s.rows = kThreads / s.cols;
  s.row_blocks = (T + s.rows - 1) / s.rows;
  s.col_blocks = whole_rows ? 1 : (groups + s.cols - 1) / s.cols;
  return s;
}

// Position of route (t, k): -1 for no route; positions outside the buffer
// are reported and skipped.
__device__ __forceinline__ int route_row(const TokensArgs& a, int64_t t, int k) {
  const int p = __ldg(a.pos + t * a.topk + k);
  if (p >= a.R) {
    raise_status(a.status, NVFP4_ERR_DEVICE_CHECK);
    return -1;
  }
  return p;
}

template <int DT, int VEC>
__device__ void zero_tail(const TokensArgs& a, int block) {
  const int n = *a.live;
  const int64_t first = n < 0 ? 0 : n;
  const int64_t groups = a.D / VEC;
  Pack<DT, VEC> z;
  z.zero();
  for (int64_t r = first + block; r < a.R; r += kTailBlocks)
    for (int64_t g = threadIdx.x; g < groups; g += kThreads) z.store(a.out, r * a.D + g * VEC);
}

template <int DT, int VEC>
__global__ void __launch_bounds__(kThreads) dispatch_rows_kernel(const TokensArgs a, int cols,
                                                                  int col_blocks, int main_blocks) {
  if (static_cast<int>(blockIdx.x) >= main_blocks) {
    zero_tail<DT, VEC>(a, blockIdx.x - main_blocks);
    return;
  }
  const int rb = blockIdx.x / col_blocks, cb = blockIdx.x % col_blocks;
  const int rows = kThreads / cols;
  const int64_t t = static_cast<int64_t>(rb) * rows + threadIdx.x / cols;
  const int64_t c = (static_cast<int64_t>(cb) * cols + threadIdx.x % cols) * VEC;
  if (t >= a.T || c >= a.D) return;
  Pack<DT, VEC> v;
  v.load(a.src, t * a.ld + c);
  for (int k = 0; k < a.topk; ++k) {
    const int p = route_row(a, t, k);
    if (p >= 0) v.store(a.out, static_cast<int64_t>(p) * a.D + c);
  }
}

template <int DT, int VEC>
__global__ void __launch_bounds__(kThreads) combine_rows_kernel(const TokensArgs a, int cols,
                                                                 int col_blocks) {
  const int rb = blockIdx.x / col_blocks, cb = blockIdx.x % col_blocks;
  const int rows = kThreads / cols;
  const int64_t t = static_cast<int64_t>(rb) * rows + threadIdx.x / cols;
  const int64_t c = (static_cast<int64_t>(cb) * cols + threadIdx.x % cols) * VEC;
  if (t >= a.T || c >= a.D) return;
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
  for (int k0 = 0; k0 < a.topk; k0 += kRoutes) {
    Pack<DT, VEC> v[kRoutes];
    int p[kRoutes];
#pragma unroll
    for (int j = 0; j < kRoutes; ++j) {
      p[j] = k0 + j < a.topk ? route_row(a, t, k0 + j) : -1;
      if (p[j] >= 0) v[j].load(a.src, static_cast<int64_t>(p[j]) * a.ld + c);
    }
#pragma unroll
    for (int j = 0; j < kRoutes; ++j) {
      if (p[j] < 0) continue;
      const float w = a.w ? __ldg(a.w + t * a.topk + k0 + j) : 1.f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] = fmaf(w, v[j].get(i), acc[i]);
    }
  }
  Pack<DT, VEC> o;
  o.from(acc);
  o.store(a.out, t * a.D + c);
}

// One group of `cols` threads per token: dy leaves as the columns go by, the
// partial dot products meet at the end (lanes, then the group's warps).
template <int DT, int VEC>
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(const TokensArgs a, int cols,
                                                                 int main_blocks) {
  __shared__ float part[kThreads / 32][kRoutes];
  if (static_cast<int>(blockIdx.x) >= main_blocks) {
    zero_tail<DT, VEC>(a, blockIdx.x - main_blocks);
    return;
  }
  const int rows = kThreads / cols;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * rows + threadIdx.x / cols;
  const int col = threadIdx.x % cols;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool on = t < a.T;
  for (int k0 = 0; k0 < a.topk; k0 += kRoutes) {
    int p[kRoutes];
    float w[kRoutes], dot[kRoutes];
#pragma unroll
    for (int j = 0; j < kRoutes; ++j) {
      const bool is = on && k0 + j < a.topk;
      p[j] = is ? route_row(a, t, k0 + j) : -1;
      w[j] = is ? __ldg(a.w + t * a.topk + k0 + j) : 0.f;
      dot[j] = 0.f;
    }
    if (on) {
      for (int64_t c = static_cast<int64_t>(col) * VEC; c < a.D; c += cols * VEC) {
        Pack<DT, VEC> d, v[kRoutes];
        d.load(a.src, t * a.ld + c);
#pragma unroll
        for (int j = 0; j < kRoutes; ++j)
          if (p[j] >= 0) v[j].load(a.y, static_cast<int64_t>(p[j]) * a.ld_y + c);
#pragma unroll
        for (int j = 0; j < kRoutes; ++j) {
          if (p[j] < 0) continue;
          float f[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            dot[j] = fmaf(d.get(i), v[j].get(i), dot[j]);
            f[i] = w[j] * d.get(i);
          }
          Pack<DT, VEC> o;
          o.from(f);
          o.store(a.out, static_cast<int64_t>(p[j]) * a.D + c);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kRoutes; ++j)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], o);
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < kRoutes; ++j) part[warp][j] = dot[j];
    }
    __syncthreads();
    if (on && col < kRoutes && k0 + col < a.topk) {
      float sum = 0.f;
      for (int i = 0; i < cols / 32; ++i) sum += part[warp + i][col];   // col < 8: first warp
      a.dw[t * a.topk + k0 + col] = sum;
    }
    __syncthreads();
  }
}

// Rows that every access finds 16-byte aligned go by 16 bytes, others by
// element.
bool wide_ok(const void* p, int64_t ld, int64_t D, int es) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * es) % 16 == 0 && (D * es) % 16 == 0;
}

// Calls f.template operator()<DT, VEC>() for the type and the access width.
template <class F>
cudaError_t by_type(int dtype, bool wide, F f) {
  switch (dtype) {
    case NVFP4_BF16:
      return wide ? f.template operator()<NVFP4_BF16, 8>() : f.template operator()<NVFP4_BF16, 1>();
    case NVFP4_FP16:
      return wide ? f.template operator()<NVFP4_FP16, 8>() : f.template operator()<NVFP4_FP16, 1>();
    default:
      return wide ? f.template operator()<NVFP4_FP32, 4>() : f.template operator()<NVFP4_FP32, 1>();
  }
}

bool fits(int64_t blocks) { return blocks <= 0x7FFFFFFFLL; }

struct LaunchDispatch {
  const TokensArgs& a;
  cudaStream_t s;
  template <int DT, int VEC> cudaError_t operator()() const {
    const Shape sh = shape_of(a.T, (a.D + VEC - 1) / VEC, false);
    const int64_t main = sh.row_blocks * sh.col_blocks;
    const int64_t blocks = main + (a.live ? kTailBlocks : 0);
    if (!fits(blocks)) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    dispatch_rows_kernel<DT, VEC><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
        a, sh.cols, static_cast<int>(sh.col_blocks), static_cast<int>(main));
    return cudaGetLastError();
  }
};

struct LaunchCombine {
  const TokensArgs& a;
  cudaStream_t s;
  template <int DT, int VEC> cudaError_t operator()() const {
    const Shape sh = shape_of(a.T, (a.D + VEC - 1) / VEC, false);
    const int64_t blocks = sh.row_blocks * sh.col_blocks;
    if (!fits(blocks)) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    combine_rows_kernel<DT, VEC><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
        a, sh.cols, static_cast<int>(sh.col_blocks));
    return cudaGetLastError();
  }
};

struct LaunchCombineGrad {
  const TokensArgs& a;
  cudaStream_t s;
  template <int DT, int VEC> cudaError_t operator()() const {
    const Shape sh = shape_of(a.T, (a.D + VEC - 1) / VEC, true);
    const int64_t blocks = sh.row_blocks + (a.live ? kTailBlocks : 0);
    if (!fits(blocks)) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    combine_grad_kernel<DT, VEC><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
        a, sh.cols, static_cast<int>(sh.row_blocks));
    return cudaGetLastError();
  }
};

int elem_size(int dtype) { return dtype == NVFP4_FP32 ? 4 : 2; }

}  // namespace

cudaError_t launch_tokens_dispatch(const TokensArgs& a, int dtype, cudaStream_t s) {
  const int es = elem_size(dtype);
  const bool wide = wide_ok(a.src, a.ld, a.D, es) && wide_ok(a.out, a.D, a.D, es);
  return by_type(dtype, wide, LaunchDispatch{a, s});
}

cudaError_t launch_tokens_combine(const TokensArgs& a, int dtype, cudaStream_t s) {
  const int es = elem_size(dtype);
  const bool wide = wide_ok(a.src, a.ld, a.D, es) && wide_ok(a.out, a.D, a.D, es);
  return by_type(dtype, wide, LaunchCombine{a, s});
}

cudaError_t launch_tokens_combine_grad(const TokensArgs& a, int dtype, cudaStream_t s) {
  const int es = elem_size(dtype);
  const bool wide = wide_ok(a.src, a.ld, a.D, es) && wide_ok(a.y, a.ld_y, a.D, es) &&
                    wide_ok(a.out, a.D, a.D, es);
  return by_type(dtype, wide, LaunchCombineGrad{a, s});
}

}  // namespace nvfp4
