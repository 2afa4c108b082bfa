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
//
// Rows move by chunks of 16 bytes.  Where a base, stride or width is no
// multiple of 16 bytes (odd widths), the rows of one buffer lie at different
// offsets within a chunk: then the chunks are the aligned ones of the row that
// is written, and a source row is read by the one or two aligned chunks that
// hold its part, shifted into place (the offset is the same for a whole row).
// By element instead, eight times the accesses took more than twice as long
// (combine of 4096 x 8 BF16 rows of 5001: 213 us, like this 92 us).
//
// Measured (of the 6.8 TB/s copy rate): dispatch of 256 x 8 rows of 6144 BF16 5.2
// us (0.81), its gradient of 8192 x 8 142 us (0.94); combine of 8192 x 8 139 us
// (0.92); combine's gradient of 4096 x 8 129 us (0.97), of 1021 x 6 FP16 rows of
// 2047 13.9 us (0.55: the shifting's instructions).
#include "rows.cuh"
#include "tokens.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kTailBlocks = 152;     // blocks that zero the rows past the live ones

// One row as memory: the 16-byte chunk that its first byte lies in, that byte's
// place there, and the offset of the chunk with its last byte.  Offsets within a
// row are 32-bit (rows of at most 2^30 bytes).
struct RowPtr {
  const char* chunk;
  int lead, last;
};

template <int DT, bool ALIGNED>
__device__ __forceinline__ RowPtr row_at(const void* base, int64_t row, int64_t ld, int D) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(base) + row * ld * elem_bytes<DT>();
  RowPtr r;
  r.lead = ALIGNED ? 0 : static_cast<int>(b & 15u);
  r.chunk = reinterpret_cast<const char*>(b - r.lead);
  r.last = (r.lead + D * elem_bytes<DT>() - 1) & ~15;
  return r;
}

// Elements of the row's first chunk that lie before the row.
template <int DT>
__device__ __forceinline__ int before(const RowPtr& r) {
  return r.lead / elem_bytes<DT>();
}

// The 16 bytes from element e of a row, as read: the one (ALIGNED) or two
// aligned chunks that hold them.  e may lie up to a chunk before or behind the
// row: chunks are held to those with at least one byte of the row, so no read
// leaves the 16-byte granules of the allocation, and what lies outside the row
// is arbitrary.  No branches: the reads of several rows are issued together and
// put in place afterwards.
template <int DT, bool ALIGNED>
struct Raw {
  uint4 lo, hi;
  uint32_t s;                        // offset within lo, bytes
  __device__ __forceinline__ void load(const RowPtr& r, int e) {
    const int off = r.lead + e * elem_bytes<DT>();
    if constexpr (ALIGNED) {
      lo = __ldg(reinterpret_cast<const uint4*>(r.chunk + off));
    } else {
      const int at = off & ~15;
      s = off & 15;
      lo = __ldg(reinterpret_cast<const uint4*>(r.chunk + min(max(at, 0), r.last)));
      hi = __ldg(reinterpret_cast<const uint4*>(r.chunk + min(at + 16, r.last)));   // at >= -16
    }
  }
  // ALIGNED alone: a chunk of a row that may begin and end within its chunks
  __device__ __forceinline__ void load_chunk(const RowPtr& r, int e) {
    const int off = r.lead + e * elem_bytes<DT>();
    lo = __ldg(reinterpret_cast<const uint4*>(r.chunk + min(max(off, 0), r.last)));
  }
  __device__ __forceinline__ Pack<DT, elems_per_16b<DT>()> get() const {
    Pack<DT, elems_per_16b<DT>()> v;
    uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if constexpr (!ALIGNED) {
#pragma unroll
      for (int i = 0; i < 6; ++i) x[i] = s & 8u ? x[i + 2] : x[i];
#pragma unroll
      for (int i = 0; i < 5; ++i) x[i] = s & 4u ? x[i + 1] : x[i];
      if constexpr (elem_bytes<DT>() == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __funnelshift_r(x[i], x[i + 1], 8 * (s & 2u));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v.w[i] = x[i];
    return v;
  }
};

// Stores a chunk at element e of a row, whose address is a chunk's: the whole
// chunk where it lies inside the row, else its elements inside the row.
template <int DT, bool ALIGNED>
__device__ __forceinline__ void store_at(const RowPtr& r, int e, int D,
                                         const Pack<DT, elems_per_16b<DT>()>& v) {
  constexpr int N = elems_per_16b<DT>();
  using Bits = typename Elem<DT>::Bits;
  Bits* p = reinterpret_cast<Bits*>(const_cast<char*>(r.chunk) + r.lead + e * elem_bytes<DT>());
  if (ALIGNED || (e >= 0 && e + N <= D)) {
    *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e + i >= 0 && e + i < D)
        p[i] = static_cast<Bits>(elem_bytes<DT>() == 4 ? v.w[i] : v.w[i >> 1] >> (16 * (i & 1)));
  }
}

// Chunks a row can take, wherever it starts.
template <int DT, bool ALIGNED>
__host__ __device__ __forceinline__ int chunks_of(int D) {
  constexpr int N = elems_per_16b<DT>();
  return ALIGNED ? D / N : (D + 2 * N - 2) / N;
}

// Chunks a thread has in flight for R routes: about eight reads, so that few
// routes do not leave a thread with little on its way (combine of 8192 x 2 FP32
// rows of 2048: 58 us with one chunk, 32 us with four); shifted rows take two
// reads a chunk and twice the registers.
template <bool ALIGNED> constexpr int chunks_in_flight(int R) { return (ALIGNED ? 8 : 4) / R; }

// A block covers `rows` tokens x `cols` chunks, times the chunks a thread
// takes (rows * cols = 256 threads); narrow rows share a block.
struct Shape {
  int cols, rows;
  int64_t row_blocks, col_blocks;
};

Shape shape_of(int64_t T, int64_t chunks, int per_thread, bool whole_rows) {
  Shape s;
  chunks = (chunks + per_thread - 1) / per_thread;
  s.cols = 32;
  while (s.cols < kThreads && s.cols < chunks) s.cols *= 2;
  s.rows = kThreads / s.cols;
  s.row_blocks = (T + s.rows - 1) / s.rows;
  s.col_blocks = whole_rows ? 1 : (chunks + s.cols - 1) / s.cols;
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

template <int DT, bool ALIGNED>
__device__ void zero_tail(const TokensArgs& a, int block) {
  constexpr int N = elems_per_16b<DT>();
  const int n = *a.live;
  const int64_t first = n < 0 ? 0 : n;
  Pack<DT, N> z;
  z.zero();
  for (int64_t r = first + block; r < a.R; r += kTailBlocks) {
    const RowPtr row = row_at<DT, ALIGNED>(a.out, r, a.D, a.D);
    for (int i = threadIdx.x; i < chunks_of<DT, ALIGNED>(a.D); i += blockDim.x)
      store_at<DT, ALIGNED>(row, i * N - before<DT>(row), a.D, z);
  }
}

template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) dispatch_rows_kernel(const TokensArgs a, int cols,
                                                                  int col_blocks, int main_blocks) {
  constexpr int N = elems_per_16b<DT>();
  if (static_cast<int>(blockIdx.x) >= main_blocks) {
    zero_tail<DT, ALIGNED>(a, blockIdx.x - main_blocks);
    return;
  }
  const int rb = blockIdx.x / col_blocks, cb = blockIdx.x % col_blocks;
  const int64_t t = static_cast<int64_t>(rb) * (kThreads / cols) + threadIdx.x / cols;
  const int i = cb * cols + threadIdx.x % cols;
  if (t >= a.T || i >= chunks_of<DT, ALIGNED>(a.D)) return;
  const RowPtr x = row_at<DT, ALIGNED>(a.src, t, a.ld, a.D);
  if constexpr (ALIGNED) {
    Raw<DT, true> raw;
    raw.load(x, i * N);
    const Pack<DT, N> v = raw.get();
    for (int k = 0; k < a.topk; ++k) {
      const int p = route_row(a, t, k);
      if (p >= 0) store_at<DT, true>(row_at<DT, true>(a.out, p, a.D, a.D), i * N, a.D, v);
    }
  } else {
    // the row is read again (from L1) for each destination's chunks
    for (int k = 0; k < a.topk; ++k) {
      const int p = route_row(a, t, k);
      if (p < 0) continue;
      const RowPtr o = row_at<DT, false>(a.out, p, a.D, a.D);
      const int e = i * N - before<DT>(o);
      if (e >= a.D) continue;
      Raw<DT, false> raw;
      raw.load(x, e);
      store_at<DT, false>(o, e, a.D, raw.get());
    }
  }
}

// R routes and U chunks a thread in flight.
template <int DT, bool ALIGNED, int R>
__global__ void __launch_bounds__(kThreads, ALIGNED && R > 2 ? 4 : 3) combine_rows_kernel(const TokensArgs a, int cols,
                                                                 int col_blocks) {
  constexpr int N = elems_per_16b<DT>();
  constexpr int U = chunks_in_flight<ALIGNED>(R);
  const int rb = blockIdx.x / col_blocks, cb = blockIdx.x % col_blocks;
  const int64_t t = static_cast<int64_t>(rb) * (kThreads / cols) + threadIdx.x / cols;
  const int i = cb * cols * U + threadIdx.x % cols;
  if (t >= a.T || i >= chunks_of<DT, ALIGNED>(a.D)) return;
  const RowPtr out = row_at<DT, ALIGNED>(a.out, t, a.D, a.D);
  const int e = i * N - before<DT>(out);
  const int step = cols * N;
  float acc[U][N];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int n = 0; n < N; ++n) acc[u][n] = 0.f;
  for (int k0 = 0; k0 < a.topk; k0 += R) {
    Raw<DT, ALIGNED> v[R][U];
    int p[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      p[j] = k0 + j < a.topk ? route_row(a, t, k0 + j) : -1;
      if (p[j] < 0) continue;
      const RowPtr y = row_at<DT, ALIGNED>(a.src, p[j], a.ld, a.D);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (e + u * step < a.D) v[j][u].load(y, e + u * step);
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (p[j] < 0) continue;
      const float w = a.w ? __ldg(a.w + t * a.topk + k0 + j) : 1.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Pack<DT, N> q = v[j][u].get();
#pragma unroll
        for (int n = 0; n < N; ++n) acc[u][n] = fmaf(w, q.get(n), acc[u][n]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (e + u * step >= a.D) break;
    Pack<DT, N> o;
    o.from(acc[u]);
    store_at<DT, ALIGNED>(out, e + u * step, a.D, o);
  }
}

// Rows on chunks: one group of `cols` threads per token, dout read once for all
// of R routes.  dy leaves as the chunks go by, the partial dot products meet at
// the end (lanes, then the group's warps).  Three blocks of 256 threads per SM:
// 138 us with two, 129 us with three (4096 x 8 BF16 rows of 6144).  Few tokens
// take blocks of 768 threads, which read a row of 6144 in one go (one token: 6.2
// us with 256).
template <int DT, int R, int TH>
__global__ void __launch_bounds__(TH, 768 / TH) combine_grad_kernel(const TokensArgs a, int cols,
                                                                    int main_blocks) {
  constexpr int N = elems_per_16b<DT>();
  constexpr int U = chunks_in_flight<true>(R);
  __shared__ float part[TH / 32][R];
  if (static_cast<int>(blockIdx.x) >= main_blocks) {
    zero_tail<DT, true>(a, blockIdx.x - main_blocks);
    return;
  }
  const int rows = TH / cols;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * rows + threadIdx.x / cols;
  const int col = threadIdx.x % cols;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool on = t < a.T;
  const int chunks = chunks_of<DT, true>(a.D);
  const RowPtr dout = row_at<DT, true>(a.src, on ? t : 0, a.ld, a.D);
  for (int k0 = 0; k0 < a.topk; k0 += R) {
    int p[R];
    float w[R], dot[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool is = on && k0 + j < a.topk;
      p[j] = is ? route_row(a, t, k0 + j) : -1;
      w[j] = is ? __ldg(a.w + t * a.topk + k0 + j) : 0.f;
      dot[j] = 0.f;
    }
    if (on) {
      for (int i0 = col; i0 < chunks; i0 += U * cols) {
        Raw<DT, true> d[U], v[U][R];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * cols;
          if (i >= chunks) break;
          d[u].load(dout, i * N);
#pragma unroll
          for (int j = 0; j < R; ++j)
            if (p[j] >= 0) v[u][j].load(row_at<DT, true>(a.y, p[j], a.ld_y, a.D), i * N);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * cols;
          if (i >= chunks) break;
          const Pack<DT, N> dq = d[u].get();
#pragma unroll
          for (int j = 0; j < R; ++j) {
            if (p[j] < 0) continue;
            const Pack<DT, N> vq = v[u][j].get();
            float f[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
              f[n] = w[j] * dq.get(n);
              dot[j] = fmaf(dq.get(n), vq.get(n), dot[j]);
            }
            Pack<DT, N> q;
            q.from(f);
            store_at<DT, true>(row_at<DT, true>(a.out, p[j], a.D, a.D), i * N, a.D, q);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], o);
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < R; ++j) part[warp][j] = dot[j];
    }
    __syncthreads();
    if (on && col < R && k0 + col < a.topk) {
      float sum = 0.f;
      for (int i = 0; i < cols / 32; ++i) sum += part[warp + i][col];   // col < R: first warp
      a.dw[t * a.topk + k0 + col] = sum;
    }
    __syncthreads();
  }
}

// Other rows: one warp per route.  dout is read (from L1 by the token's other
// warps) and put in place for each route's chunks.  SAME: every row of y begins
// at the same place within a chunk as its row of dy (both dense), so that only
// dout is shifted.
template <int DT, bool SAME>
__global__ void __launch_bounds__(kThreads) combine_grad_shifted_kernel(const TokensArgs a,
                                                                         int main_blocks) {
  constexpr int N = elems_per_16b<DT>();
  constexpr int U = 4;
  if (static_cast<int>(blockIdx.x) >= main_blocks) {
    zero_tail<DT, false>(a, blockIdx.x - main_blocks);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int64_t g = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = g / a.topk;
  if (t >= a.T) return;
  const int p = route_row(a, t, static_cast<int>(g - t * a.topk));
  if (p < 0) {
    if (lane == 0) a.dw[g] = 0.f;
    return;
  }
  const float w = __ldg(a.w + g);
  const RowPtr dout = row_at<DT, false>(a.src, t, a.ld, a.D);
  const RowPtr y = row_at<DT, false>(a.y, p, a.ld_y, a.D);
  const RowPtr out = row_at<DT, false>(a.out, p, a.D, a.D);
  float dot = 0.f;
  for (int e0 = lane * N - before<DT>(out); e0 < a.D; e0 += U * 32 * N) {
    Raw<DT, false> d[U];
    Raw<DT, SAME> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = e0 + u * 32 * N;
      if (e >= a.D) break;
      d[u].load(dout, e);
      if constexpr (SAME) v[u].load_chunk(y, e);
      else v[u].load(y, e);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = e0 + u * 32 * N;
      if (e >= a.D) break;
      const Pack<DT, N> dq = d[u].get(), vq = v[u].get();
      float f[N];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        f[n] = w * dq.get(n);
        if (e + n >= 0 && e + n < a.D) dot = fmaf(dq.get(n), vq.get(n), dot);
      }
      Pack<DT, N> q;
      q.from(f);
      store_at<DT, false>(out, e, a.D, q);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
  if (lane == 0) a.dw[g] = dot;
}

// Rows that every access finds on 16-byte chunks.
bool on_chunks(const void* p, int64_t ld, int64_t D, int es) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * es) % 16 == 0 && (D * es) % 16 == 0;
}

// Calls f.template operator()<DT, ALIGNED>() for the type.
template <class F>
cudaError_t by_type(int dtype, bool aligned, F f) {
  switch (dtype) {
    case NVFP4_BF16:
      return aligned ? f.template operator()<NVFP4_BF16, true>()
                     : f.template operator()<NVFP4_BF16, false>();
    case NVFP4_FP16:
      return aligned ? f.template operator()<NVFP4_FP16, true>()
                     : f.template operator()<NVFP4_FP16, false>();
    default:
      return aligned ? f.template operator()<NVFP4_FP32, true>()
                     : f.template operator()<NVFP4_FP32, false>();
  }
}

bool fits(int64_t blocks) { return blocks <= 0x7FFFFFFFLL; }

struct LaunchDispatch {
  const TokensArgs& a;
  cudaStream_t s;
  template <int DT, bool ALIGNED> cudaError_t operator()() const {
    const Shape sh = shape_of(a.T, chunks_of<DT, ALIGNED>(a.D), 1, false);
    const int64_t main = sh.row_blocks * sh.col_blocks;
    const int64_t blocks = main + (a.live ? kTailBlocks : 0);
    if (!fits(blocks)) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    dispatch_rows_kernel<DT, ALIGNED><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
        a, sh.cols, static_cast<int>(sh.col_blocks), static_cast<int>(main));
    return cudaGetLastError();
  }
};

struct LaunchCombine {
  const TokensArgs& a;
  cudaStream_t s;
  template <int DT, bool ALIGNED> cudaError_t operator()() const {
    if (a.topk <= 2) return go<DT, ALIGNED, 2>();
    if (!ALIGNED || a.topk <= 4) return go<DT, ALIGNED, 4>();
    return go<DT, true, 8>();
  }
  template <int DT, bool ALIGNED, int R> cudaError_t go() const {
    const Shape sh =
        shape_of(a.T, chunks_of<DT, ALIGNED>(a.D), chunks_in_flight<ALIGNED>(R), false);
    const int64_t blocks = sh.row_blocks * sh.col_blocks;
    if (!fits(blocks)) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    combine_rows_kernel<DT, ALIGNED, R><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
        a, sh.cols, static_cast<int>(sh.col_blocks));
    return cudaGetLastError();
  }
};

struct LaunchCombineGrad {
  const TokensArgs& a;
  cudaStream_t s;
  bool same;
  template <int DT, bool ALIGNED> cudaError_t operator()() const {
    if constexpr (ALIGNED) {
      if (a.topk <= 2) return rows<DT, 2>();
      return a.topk <= 4 ? rows<DT, 4>() : rows<DT, 8>();
    } else {
      return same ? shifted<DT, true>() : shifted<DT, false>();
    }
  }
  template <int DT, int R> cudaError_t rows() const {
    const Shape sh = shape_of(a.T, chunks_of<DT, true>(a.D), chunks_in_flight<true>(R), true);
    const int64_t blocks = sh.row_blocks + (a.live ? kTailBlocks : 0);
    if (!fits(blocks)) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    const unsigned g = static_cast<unsigned>(blocks);
    // one block per SM or less, and rows that 256 threads do not cover
    if (sh.cols == kThreads && sh.row_blocks <= kTailBlocks)
      combine_grad_kernel<DT, R, 768><<<g, 768, 0, s>>>(a, 768, static_cast<int>(sh.row_blocks));
    else
      combine_grad_kernel<DT, R, kThreads><<<g, kThreads, 0, s>>>(a, sh.cols,
                                                                 static_cast<int>(sh.row_blocks));
    return cudaGetLastError();
  }
  template <int DT, bool SAME> cudaError_t shifted() const {
    const int64_t main = (a.T * a.topk + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t blocks = main + (a.live ? kTailBlocks : 0);
    if (!fits(blocks)) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    combine_grad_shifted_kernel<DT, SAME><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
        a, static_cast<int>(main));
    return cudaGetLastError();
  }
};

int elem_size(int dtype) { return dtype == NVFP4_FP32 ? 4 : 2; }

}  // namespace

cudaError_t launch_tokens_dispatch(const TokensArgs& a, int dtype, cudaStream_t s) {
  const int es = elem_size(dtype);
  const bool aligned = on_chunks(a.src, a.ld, a.D, es) && on_chunks(a.out, a.D, a.D, es);
  return by_type(dtype, aligned, LaunchDispatch{a, s});
}

cudaError_t launch_tokens_combine(const TokensArgs& a, int dtype, cudaStream_t s) {
  const int es = elem_size(dtype);
  const bool aligned = on_chunks(a.src, a.ld, a.D, es) && on_chunks(a.out, a.D, a.D, es);
  return by_type(dtype, aligned, LaunchCombine{a, s});
}

cudaError_t launch_tokens_combine_grad(const TokensArgs& a, int dtype, cudaStream_t s) {
  const int es = elem_size(dtype);
  const bool aligned = on_chunks(a.src, a.ld, a.D, es) && on_chunks(a.y, a.ld_y, a.D, es) &&
                       on_chunks(a.out, a.D, a.D, es);
  const bool same = a.ld_y == a.D && ((reinterpret_cast<uintptr_t>(a.y) ^
                                       reinterpret_cast<uintptr_t>(a.out)) & 15u) == 0;
  return by_type(dtype, aligned, LaunchCombineGrad{a, s, same});
}

}  // namespace nvfp4
