// Root-mean-square norm with the residual's addition, and its gradient:
//
//   h = x + r                     rounded to the rows' type: it is an output, and
//                                 what the gradient is taken at
//   y = h * rstd * w              rstd = 1 / sqrt(mean(h^2) + eps)
//   dx = rstd (g - h rstd^2 mean(g h)) + dh,   g = dy w
//   dw = sum_t dy h rstd
//
// One pass: a row stays in its threads' registers between the reduction and the
// products, so every byte moves once.  The output is y in the rows' type or, for the
// FP8 products, E4M3 codes with one scale per 128 columns, taken from the unrounded
// y (one rounding).  A thread holds 8 or 16 elements of a row and rows share a
// block where they are narrow; rows whose bases, strides or width are no multiple of
// 16 bytes move element by element, neighbouring threads on neighbouring elements.
//
// dw: each block keeps its rows' sums in registers (a thread has the same columns of
// every row), writes them once, and a second launch adds the blocks' in order.  No
// atomics: results repeat bit for bit.  Sums are FP32.  Bound: HBM.
#include "fp8_quant.cuh"
#include "norm.h"

namespace nvfp4 {

namespace {

constexpr int kSms = 152;                 // the workspace's size hangs on it

// Threads of a row, and rows of a block.
struct NormShape {
  int ept, threads, rows;
};

// The sum over a row's threads of N values, the same in each of them: lanes, then warps
// in shared memory (which calls of one kernel share: a barrier first).
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int threads, float (*part)[N]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if (threads == 32) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = threads >> 5, first = warp / warps * warps;
  __syncthreads();
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) part[warp][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < warps ? part[first + lane][i] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
}

__device__ __forceinline__ float weight_at(const void* w, int type, int c) {
  if (type == NVFP4_FP32) return __ldg(static_cast<const float*>(w) + c);
  const uint32_t b = __ldg(static_cast<const uint16_t*>(w) + c);
  return type == NVFP4_BF16 ? elem_to_f32<NVFP4_BF16>(b) : elem_to_f32<NVFP4_FP16>(b);
}

// VEC weights from column c on (base aligned to 16 bytes where VEC > 1).
template <int VEC>
__device__ __forceinline__ void load_weights(const void* w, int type, int c, float* f) {
  if constexpr (VEC == 1) {
    f[0] = weight_at(w, type, c);
  } else if (type == NVFP4_FP32) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + c + i));
      f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
    }
  } else if constexpr (VEC == 8) {
    if (type == NVFP4_BF16) {
      Pack<NVFP4_BF16, 8> p;
      p.load(w, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = p.get(i);
    } else {
      Pack<NVFP4_FP16, 8> p;
      p.load(w, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = p.get(i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = weight_at(w, type, c + i);
  }
}

template <int DT, int VEC>
__device__ __forceinline__ void store(void* base, int64_t at, const Pack<DT, VEC>& p) {
  using Bits = typename Elem<DT>::Bits;
  Bits* d = static_cast<Bits*>(base) + at;
  if constexpr (VEC == 1) *d = static_cast<Bits>(p.w[0]);
  else *reinterpret_cast<uint4*>(d) = make_uint4(p.w[0], p.w[1], p.w[2], p.w[3]);
}

template <int DT, int VEC, int EPT, bool FP8, int MOST>
__global__ void __launch_bounds__(MOST) rms_norm_kernel(const NormArgs a, int threads, int rows) {
  constexpr int V = EPT / VEC;
  __shared__ float part[32][1];
  const int sub = threadIdx.x / threads, tid = threadIdx.x - sub * threads;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * rows + sub;
  const bool on = row < a.T;
  Pack<DT, VEC> px[V], pr[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * threads + tid) * VEC;
    px[i].zero();
    pr[i].zero();
    if (on && c < a.D) {
      px[i].load(a.x, row * a.ld + c);
      if (a.r) pr[i].load(a.r, row * a.ld_r + c);
    }
  }
  float w[EPT], h[EPT], sum[1] = {0.f};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * threads + tid) * VEC;
    if (c < a.D) {
      load_weights<VEC>(a.w, a.w_type, c, w + i * VEC);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) w[i * VEC + j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (a.r) {
      float f[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = px[i].get(j) + pr[i].get(j);
      px[i].from(f);
      const int c = (i * threads + tid) * VEC;
      if (on && c < a.D) store<DT, VEC>(a.h, row * a.D + c, px[i]);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float f = px[i].get(j);
      h[i * VEC + j] = f;
      sum[0] = fmaf(f, f, sum[0]);
    }
  }
  row_sum<1>(sum, threads, part);
  const float rstd = 1.f / sqrtf(sum[0] / static_cast<float>(a.D) + a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * threads + tid) * VEC;
    float y[VEC];
    if constexpr (FP8) {
      // The quotient 448 y / max |y| does not hold rstd: it is taken from the products
      // h w (exact for 16-bit factors), so that codes are rounded from the real quotient
      // also next to a border; with rstd only where a maximum leaves the normal range.
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        y[j] = h[i * VEC + j] * w[i * VEC + j];
        amax = fmaxf(amax, fabsf(y[j]));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
      const bool direct = amax >= kAmaxFloor && amax * rstd >= kAmaxFloor && amax < INFINITY;
      if (!direct) {
        amax = 0.f;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          y[j] = h[i * VEC + j] * rstd * w[i * VEC + j];
          amax = fmaxf(amax, fabsf(y[j]));
        }
      }
      // (`direct` is the same in the 16 lanes of a block, not in the warp's two blocks)
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
      if (on && c < a.D) {
        const BlockScale32 b(amax);
        uint2 q;
        q.x = e4m3x4(b.quotient(y[0]), b.quotient(y[1]), b.quotient(y[2]), b.quotient(y[3]));
        q.y = e4m3x4(b.quotient(y[4]), b.quotient(y[5]), b.quotient(y[6]), b.quotient(y[7]));
        *reinterpret_cast<uint2*>(a.codes + row * a.D + c) = q;
        if ((c & 127) == 0)
          a.scales[static_cast<int64_t>(c >> 7) * a.T + row] = direct ? b.scale * rstd : b.scale;
      }
    } else if (on && c < a.D) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) y[j] = h[i * VEC + j] * rstd * w[i * VEC + j];
      Pack<DT, VEC> p;
      p.from(y);
      store<DT, VEC>(a.y, row * a.D + c, p);
    }
  }
}

template <int DT, int VEC, int EPT, int MOST>
__global__ void __launch_bounds__(MOST) rms_norm_grad_kernel(const NormArgs a, int threads,
                                                             int rows) {
  constexpr int V = EPT / VEC;
  __shared__ float part[32][2];
  const int sub = threadIdx.x / threads, tid = threadIdx.x - sub * threads;
  float w[EPT], dw[EPT];
#pragma unroll
  for (int i = 0; i < EPT; ++i) w[i] = dw[i] = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * threads + tid) * VEC;
    if (c < a.D) load_weights<VEC>(a.w, a.w_type, c, w + i * VEC);
  }
  const float over = 1.f / static_cast<float>(a.D);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rows; base < a.T;
       base += static_cast<int64_t>(gridDim.x) * rows) {
    const int64_t row = base + sub;
    const bool on = row < a.T;
    Pack<DT, VEC> ph[V], pd[V], pr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * threads + tid) * VEC;
      ph[i].zero();
      pd[i].zero();
      pr[i].zero();
      if (on && c < a.D) {
        ph[i].load(a.x, row * a.ld + c);
        pd[i].load(a.dy, row * a.ld_dy + c);
        if (a.r) pr[i].load(a.r, row * a.ld_r + c);
      }
    }
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float h = ph[i].get(j);
        sum[0] = fmaf(h, h, sum[0]);
        sum[1] = fmaf(pd[i].get(j) * w[i * VEC + j], h, sum[1]);
      }
    row_sum<2>(sum, threads, part);
    const float rstd = 1.f / sqrtf(sum[0] * over + a.eps);
    const float back = rstd * rstd * (sum[1] * over);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * threads + tid) * VEC;
      float f[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float h = ph[i].get(j), d = pd[i].get(j);
        f[j] = rstd * fmaf(d, w[i * VEC + j], -h * back) + pr[i].get(j);
        dw[i * VEC + j] = fmaf(d, h * rstd, dw[i * VEC + j]);
      }
      if (on && c < a.D) {
        Pack<DT, VEC> p;
        p.from(f);
        store<DT, VEC>(a.y, row * a.D + c, p);
      }
    }
  }
  float* out = a.part + (static_cast<int64_t>(blockIdx.x) * rows + sub) * a.D;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * threads + tid) * VEC;
    if (c < a.D) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) out[c + j] = dw[i * VEC + j];
    }
  }
}

// dw[c] = sum of the parts' column c: 32 columns a block, 32 warps on every 32nd part.
__global__ void __launch_bounds__(1024) rms_norm_dw_kernel(const float* part, int parts, int D,
                                                           int type, void* dw) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < D)
    for (int p = warp; p < parts; p += 32) v += part[static_cast<int64_t>(p) * D + c];
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < D) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sums[i][lane];
    if (type == NVFP4_FP32) static_cast<float*>(dw)[c] = v;
    else static_cast<uint16_t*>(dw)[c] = static_cast<uint16_t>(
        type == NVFP4_BF16 ? f32_to_elem<NVFP4_BF16>(v) : f32_to_elem<NVFP4_FP16>(v));
  }
}

// Elements a thread takes of a row: 8 while there are few rows (a row's time is then
// its latency) or a row has few elements, 16 where rows fill the SMs anyway.
NormShape shape_of(int64_t T, int64_t D) {
  NormShape s{};
  s.ept = (T > 2 * kSms && D > 32 * 4 * 8) || D > 1024 * 8 ? 16 : 8;
  s.threads = static_cast<int>((D + 32 * s.ept - 1) / (32 * s.ept)) * 32;
  s.rows = s.threads >= 256 ? 1 : 256 / s.threads;
  return s;
}

bool vectors(const NormArgs& a, int dtype, bool grad) {
  const int es = dtype == NVFP4_FP32 ? 4 : 2;
  auto row16 = [&](const void* p, int64_t ld) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (a.T <= 1 || ld * es % 16 == 0));
  };
  return static_cast<int64_t>(a.D) * es % 16 == 0 && row16(a.x, a.ld) && row16(a.r, a.ld_r) &&
         row16(a.w, 0) && row16(a.h, a.D) && row16(a.y, a.D) && (!grad || row16(a.dy, a.ld_dy));
}

template <int DT, int VEC, bool FP8>
cudaError_t forward(const NormArgs& a, const NormShape& s, cudaStream_t st) {
  const int64_t blocks = (a.T + s.rows - 1) / s.rows;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  const unsigned g = static_cast<unsigned>(blocks), n = static_cast<unsigned>(s.threads * s.rows);
  if (s.ept == 8) rms_norm_kernel<DT, VEC, 8, FP8, 1024><<<g, n, 0, st>>>(a, s.threads, s.rows);
  else if (n <= 512) rms_norm_kernel<DT, VEC, 16, FP8, 512><<<g, n, 0, st>>>(a, s.threads, s.rows);
  else rms_norm_kernel<DT, VEC, 16, FP8, 1024><<<g, n, 0, st>>>(a, s.threads, s.rows);
  return cudaGetLastError();
}

int grad_blocks(int64_t T, const NormShape& s) {
  const int64_t want = (T + s.rows - 1) / s.rows;
  const int64_t most = static_cast<int64_t>(kSms) * (s.threads * s.rows > 512 ? 1 : 2);
  return static_cast<int>(want < most ? want : most);
}

template <int DT, int VEC>
cudaError_t backward(const NormArgs& a, cudaStream_t st) {
  const NormShape s = shape_of(a.T, a.D);
  const unsigned g = static_cast<unsigned>(grad_blocks(a.T, s));
  const unsigned n = static_cast<unsigned>(s.threads * s.rows);
  if (g > 0) {
    if (s.ept == 8)
      rms_norm_grad_kernel<DT, VEC, 8, 1024><<<g, n, 0, st>>>(a, s.threads, s.rows);
    else if (n <= 512)
      rms_norm_grad_kernel<DT, VEC, 16, 512><<<g, n, 0, st>>>(a, s.threads, s.rows);
    else
      rms_norm_grad_kernel<DT, VEC, 16, 1024><<<g, n, 0, st>>>(a, s.threads, s.rows);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  rms_norm_dw_kernel<<<(a.D + 31) / 32, 1024, 0, st>>>(a.part, static_cast<int>(g) * s.rows, a.D,
                                                       a.w_type, a.dw);
  return cudaGetLastError();
}

template <int DT>
cudaError_t by_vector(const NormArgs& a, bool fp8, cudaStream_t st) {
  const NormShape s = shape_of(a.T, a.D);
  if constexpr (DT != NVFP4_FP32)
    if (fp8) return forward<DT, 8, true>(a, s, st);
  return vectors(a, DT, false) ? forward<DT, elems_per_16b<DT>(), false>(a, s, st)
                               : forward<DT, 1, false>(a, s, st);
}

}  // namespace

int norm_grad_parts(int64_t T, int64_t D) {
  const NormShape s = shape_of(T, D);
  return grad_blocks(T, s) * s.rows;
}

cudaError_t launch_rms_norm(const NormArgs& a, int dtype, bool fp8, cudaStream_t s) {
  if (dtype == NVFP4_BF16) return by_vector<NVFP4_BF16>(a, fp8, s);
  if (dtype == NVFP4_FP16) return by_vector<NVFP4_FP16>(a, fp8, s);
  return by_vector<NVFP4_FP32>(a, fp8, s);
}

cudaError_t launch_rms_norm_grad(const NormArgs& a, int dtype, cudaStream_t s) {
  const bool v = vectors(a, dtype, true);
  if (dtype == NVFP4_BF16) return v ? backward<NVFP4_BF16, 8>(a, s) : backward<NVFP4_BF16, 1>(a, s);
  if (dtype == NVFP4_FP16) return v ? backward<NVFP4_FP16, 8>(a, s) : backward<NVFP4_FP16, 1>(a, s);
  return v ? backward<NVFP4_FP32, 4>(a, s) : backward<NVFP4_FP32, 1>(a, s);
}

}  // namespace nvfp4
