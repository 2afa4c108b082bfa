// Root-mean-square norm with the residual's addition, and its gradient:
//
//   h = x + r                     rounded to the rows' type: it is an output, and
//                                 what the gradient is taken at
//   y = h * rstd * w              rstd = 1 / sqrt(mean(h^2) + eps)
//   dx = rstd (g - h rstd^2 mean(g h)) + dh,   g = dy w
//   dw = sum_t dy h rstd
//
// One pass: a row stays in its threads' registers between the reduction and the products,
// so every byte moves once.  The output is y in the rows' type or, for the FP8 products,
// E4M3 codes with one scale per 128 columns, taken from the unrounded y (one rounding).
//
// Blocks walk the rows.  A thread holds 8, 16 or 32 elements of one, in chunks of 16 bytes,
// and copies its chunks of the next rows to shared memory meanwhile (asynchronous copies
// that only it, or its warp, reads: no barrier), two rows on their way (four were no faster,
// with a residual or without).  With one row at a time an SM had 24 KB on its way: 8192 rows
// of 6144 BF16 took 51 us, now 41, their gradient with dh 126 us, now 74.  Narrow rows share a
// block.
//
// Where rows are no multiple of 16 bytes apart, chunks are the aligned ones of memory: all
// tensors of a call have their rows at the same offset in a chunk (the first and last chunk
// of a row are masked), and a block's rows are eight apart or a multiple, so that they all
// start at the same offset and the block's weights stay in registers there too.
//
// dw: each block keeps its rows' sums in registers (a thread has the same columns of
// every row), writes them once, and a second launch adds the blocks' in order.  No
// atomics: results repeat bit for bit.  Sums are FP32.
//
// Bound: HBM.  8192 x 6144 BF16, and its part of the measured copy rate: norm 41 us (0.73: a
// row's latency, of copies, sums and stores, on the 24 warps that the registers leave room
// for; FP32 rows, twice the bytes, 65 us, 0.91), with residual 65 us (0.91), codes with
// residual 61 us (0.85), gradient 68 us (0.66), with dh 73 us (0.81).  8192 x 6143: 57, 79, -,
// 81 and 91 us (masks, and weights by the element).  One row: 2.8 to 3.3 us, the gradient 3.6,
// of two rows and more 5.3 (its second launch): latency.  In a graph, one call after the other.
#include "fp8_quant.cuh"
#include "norm.h"

namespace nvfp4 {

namespace {

constexpr int kSms = 152;                 // the workspace's size hangs on it
constexpr int kNormSmem = 200 * 1024;     // of an SM for the rows on their way
// The widest FP32 gradient begun inside a chunk: 17 warps, three arrays, one row on its way.
constexpr int kNormSmemMost = 17 * 32 * 32 * 4 * 3;

// Threads of a row, rows of a block, rows on their way.
struct NormShape {
  int ept, threads, rows, depth, grid;
  size_t smem;
};
constexpr int kMostDepth = 2;
// (with or without dh the same shape: the workspace's size hangs on it)
constexpr int kGradArrays = 3;
// Registers a thread of 16 elements, and of 32.
constexpr int kForwardRegs = 80, kOddRegs = 72, kFp8Regs = 80, kGradRegs = 128;
constexpr int kWideRegs = 96, kWideFp8Regs = 128, kWideGradRegs = 128;

// The sum over a row's threads of N values, the same in each of them: lanes, then warps
// in shared memory.  `part` alternates between two places from row to row: who writes one
// again has passed the other's barrier, which everybody reaches after reading the first.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int threads, float (*part)[N]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if (threads == 32) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = threads >> 5, first = warp / warps * warps;
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

// A chunk of floats in the rows' type, two per conversion.
template <int DT, int N>
__device__ __forceinline__ void pack(Pack<DT, N>& p, const float (&f)[N]) {
  if constexpr (DT == NVFP4_FP32) {
    p.from(f);
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if constexpr (DT == NVFP4_BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p.w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
      else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(p.w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    }
  }
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  const int n = in ? 16 : 0;                        // the rest of the 16 bytes: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the latest n groups.
__device__ __forceinline__ void cp_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}

// A thread's chunks of a row: DT's type, EPT elements, the chunks next to each other
// (TOGETHER) or a row's threads apart.  Without ALIGNED a row starts `lead` elements after
// the start of its first chunk.  Copies take neighbouring chunks by neighbouring lanes also
// where a thread's own chunks lie together: its warp's lanes then copy for each other (own
// chunks by their lane took every sector of memory twice: codes of 8192 x 6144 85 -> 61 us).
template <int DT, int EPT, bool TOGETHER, bool ALIGNED>
struct Chunks {
  static constexpr int N = elems_per_16b<DT>(), V = EPT / N;
  int threads, tid, D, lead;
  __device__ __forceinline__ int column(int i) const {       // may be negative without ALIGNED
    const int c = TOGETHER ? tid * V + i : i * threads + tid;
    return c * N - (ALIGNED ? 0 : lead);
  }
  __device__ __forceinline__ bool any(int i) const { return column(i) < D; }
  __device__ __forceinline__ bool whole(int i) const {
    return ALIGNED || (column(i) >= 0 && column(i) + N <= D);
  }
  __device__ __forceinline__ bool in(int i, int j) const {
    return ALIGNED || (column(i) + j >= 0 && column(i) + j < D);
  }
  // Places of the chunk that a thread copies, and of its own, in the block's part for a row.
  __device__ __forceinline__ int copied(int i) const {
    return TOGETHER ? (tid & ~31) * V + i * 32 + (tid & 31) : i * threads + tid;
  }
  __device__ __forceinline__ uint32_t place(int chunk) const {
    return (static_cast<int>(threadIdx.x) - tid) * V * 16 + chunk * 16;
  }
  // A row's copies to shared memory.
  __device__ __forceinline__ void copy(uint32_t dst, const void* base, int64_t ld, int64_t row,
                                       bool on) const {
    const char* p = static_cast<const char*>(base) + row * ld * elem_bytes<DT>();
    // (an address of 16 bytes also where nothing is read)
    const char* none = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(base) &
                                                     ~static_cast<uintptr_t>(15));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int column = copied(i) * N - (ALIGNED ? 0 : lead);
      const bool go = on && column < D;
      cp16(dst + place(copied(i)), go ? p + column * elem_bytes<DT>() : none, go);
    }
  }
  __device__ __forceinline__ void take(uint32_t src, int i, Pack<DT, N>& p) const {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(p.w[0]), "=r"(p.w[1]), "=r"(p.w[2]), "=r"(p.w[3])
                 : "r"(src + place(TOGETHER ? tid * V + i : i * threads + tid)) : "memory");
    if (!whole(i)) {                                // what lies outside the row is not the row's
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if constexpr (N == 4) {
          if (!in(i, w)) p.w[w] = 0u;
        } else {
          p.w[w] &= (in(i, 2 * w) ? 0xFFFFu : 0u) | (in(i, 2 * w + 1) ? 0xFFFF0000u : 0u);
        }
      }
    }
  }
  __device__ __forceinline__ void take(uint32_t src, Pack<DT, N> (&p)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) take(src, i, p[i]);
  }
  __device__ __forceinline__ void put(void* base, int64_t row, int i, const Pack<DT, N>& p) const {
    using Bits = typename Elem<DT>::Bits;
    Bits* d = static_cast<Bits*>(base) + row * D + column(i);
    if (whole(i)) {
      *reinterpret_cast<uint4*>(d) = make_uint4(p.w[0], p.w[1], p.w[2], p.w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (in(i, j)) d[j] = static_cast<Bits>(N == 4 ? p.w[j & 3] : p.w[j >> 1] >> (16 * (j & 1)));
    }
  }
  __device__ __forceinline__ void weights(const void* w, int type, float (&f)[EPT]) const {
    const bool vectors = ALIGNED && (reinterpret_cast<uintptr_t>(w) & 15u) == 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = column(i);
      if (vectors && any(i)) {
        if (type == NVFP4_FP32) {
#pragma unroll
          for (int j = 0; j < N; j += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + c + j));
            f[i * N + j] = v.x; f[i * N + j + 1] = v.y;
            f[i * N + j + 2] = v.z; f[i * N + j + 3] = v.w;
          }
        } else if constexpr (DT != NVFP4_FP32) {
          Pack<DT, N> v;                            // the rows' type
          v.load(w, c);
#pragma unroll
          for (int j = 0; j < N; ++j) f[i * N + j] = v.get(j);
        }
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
          f[i * N + j] = any(i) && in(i, j) ? weight_at(w, type, c + j) : 0.f;
      }
    }
  }
};

template <int DT>
__device__ __forceinline__ int lead_of(const void* base, int64_t ld, int64_t row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(base) + row * ld * elem_bytes<DT>()) & 15u) /
         elem_bytes<DT>();
}

template <int DT, int EPT, bool FP8, bool ALIGNED, int REGS>
__global__ void __maxnreg__(REGS) rms_norm_kernel(const NormArgs a, int threads, int rows,
                                                  int depth) {
  using C = Chunks<DT, EPT, FP8, ALIGNED>;
  constexpr int N = C::N, V = C::V;
  extern __shared__ uint4 staged[];                 // [depth][arrays][V][threads of the block]
  __shared__ float part[2][32][1];
  const int sub = threadIdx.x / threads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * rows;
  const C c{threads, static_cast<int>(threadIdx.x) - sub * threads, a.D,
            ALIGNED ? 0 : lead_of<DT>(a.x, a.ld, first + sub)};
  const int arrays = a.r ? 2 : 1;
  const uint32_t all = smem_u32(staged), size = blockDim.x * V * 16;
  auto place = [&](int slot, int array) { return all + (slot * arrays + array) * size; };
  auto copy = [&](int64_t base, int slot) {
    const int64_t row = base + sub;
    c.copy(place(slot, 0), a.x, a.ld, row, row < a.T);
    if (a.r) c.copy(place(slot, 1), a.r, a.ld_r, row, row < a.T);
    cp_commit();
  };
  for (int i = 0; i < depth; ++i) copy(first + i * step, i);
  float w[EPT];
  c.weights(a.w, a.w_type, w);
  int slot = 0, odd = 0;
#pragma unroll 1
  for (int64_t base = first; base < a.T; base += step) {
    const int64_t row = base + sub;
    const bool on = row < a.T;
    cp_wait(depth - 1);
    if constexpr (FP8) __syncwarp();                // other lanes' copies
    Pack<DT, N> px[V];
    c.take(place(slot, 0), px);
    float sum[1] = {0.f};
    if (a.r) {
      Pack<DT, N> pr[V];
      c.take(place(slot, 1), pr);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float f[N];
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] = px[i].get(j) + pr[i].get(j);
        pack<DT, N>(px[i], f);
        if (on && c.any(i)) c.put(a.h, row, i, px[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) sum[0] = fmaf(px[i].get(j), px[i].get(j), sum[0]);
    row_sum<1>(sum, threads, part[odd]);
    odd ^= 1;
    if constexpr (FP8) __syncwarp();
    copy(base + depth * step, slot);                // the slot has been read
    if (++slot == depth) slot = 0;
    const float rstd = 1.f / sqrtf(sum[0] / static_cast<float>(a.D) + a.eps);
    if constexpr (FP8) {
      // The quotient 448 y / max |y| does not hold rstd: it is taken from the products h w
      // (exact for 16-bit factors), so that codes are rounded from the real quotient also
      // next to a border; with rstd only where a maximum leaves the normal range.  For BF16
      // factors the products have 16 bits, a border times the maximum 21, so a quotient
      // meets a border or misses it by 2^-21 of its value, and BlockScale's, good to 2^-23,
      // will do.
      constexpr int kLanes = 128 / EPT;             // of a block of 128 columns
      float y[EPT], amax = 0.f;
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        y[j] = px[j / N].get(j % N) * w[j];
        amax = fmaxf(amax, fabsf(y[j]));
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
      const bool direct = amax >= kAmaxFloor && amax * rstd >= kAmaxFloor && amax < INFINITY;
      if (!__all_sync(0xFFFFFFFFu, direct)) {
        float again = 0.f;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
          if (!direct) y[j] = px[j / N].get(j % N) * rstd * w[j];
          again = fmaxf(again, fabsf(y[j]));
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
          again = fmaxf(again, __shfl_xor_sync(0xFFFFFFFFu, again, o));
        amax = again;
      }
      const int col = c.column(0);
      if (on && col < a.D) {                        // D % 16 == 0: whole sixteens
        uint32_t q[EPT / 4];
        float scale;
        auto codes = [&](const auto& b) {
          scale = b.scale;
#pragma unroll
          for (int j = 0; j < EPT / 4; ++j)
            q[j] = e4m3x4(b.quotient(y[4 * j]), b.quotient(y[4 * j + 1]),
                          b.quotient(y[4 * j + 2]), b.quotient(y[4 * j + 3]));
        };
        if (DT == NVFP4_BF16 && a.w_type == NVFP4_BF16 && direct) codes(BlockScale(amax));
        else codes(BlockScale32(amax));
        uint8_t* out = a.codes + row * a.D + col;
        if constexpr (EPT == 8) {
          *reinterpret_cast<uint2*>(out) = make_uint2(q[0], q[1]);
        } else {
#pragma unroll
          for (int j = 0; j < EPT / 16; ++j)
            if (col + 16 * j < a.D)
              *reinterpret_cast<uint4*>(out + 16 * j) =
                  make_uint4(q[4 * j], q[4 * j + 1], q[4 * j + 2], q[4 * j + 3]);
        }
        if ((col & 127) == 0)
          a.scales[static_cast<int64_t>(col >> 7) * a.T + row] = direct ? scale * rstd : scale;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (on && c.any(i)) {
          float y[N];
#pragma unroll
          for (int j = 0; j < N; ++j) y[j] = px[i].get(j) * rstd * w[i * N + j];
          Pack<DT, N> p;
          pack<DT, N>(p, y);
          c.put(a.y, row, i, p);
        }
      }
    }
  }
  cp_wait(0);
}

__device__ __forceinline__ void put_dw(void* dw, int type, int col, float v) {
  if (type == NVFP4_FP32) static_cast<float*>(dw)[col] = v;
  else static_cast<uint16_t*>(dw)[col] = static_cast<uint16_t>(
      type == NVFP4_BF16 ? f32_to_elem<NVFP4_BF16>(v) : f32_to_elem<NVFP4_FP16>(v));
}

template <int DT, int EPT, bool ALIGNED, int REGS>
__global__ void __maxnreg__(REGS) rms_norm_grad_kernel(const NormArgs a, int threads, int rows,
                                                       int depth) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using C = Chunks<DT, EPT, false, ALIGNED>;
  constexpr int N = C::N, V = C::V;
  // dh is taken with the others, so that the slot's next copies start at once (8192 x 6144
  // 78 -> 74 us); masked chunks take it behind the sums, when fewer registers are in use (8192
  // x 6143 97 -> 91 us).  32 elements a thread and their weights and sums leave no registers
  // for a row: it is read from shared memory again behind the sums (4096 x 12288 216 -> 78 us).
  constexpr bool kKept = EPT < 32, kEarly = ALIGNED && kKept;
  extern __shared__ uint4 staged[];
  __shared__ float part[2][32][2];
  const int sub = threadIdx.x / threads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * rows;
  const C c{threads, static_cast<int>(threadIdx.x) - sub * threads, a.D,
            ALIGNED ? 0 : lead_of<DT>(a.x, a.ld, first + sub)};
  const int arrays = a.r ? 3 : 2;
  const uint32_t all = smem_u32(staged), size = blockDim.x * V * 16;
  auto place = [&](int slot, int array) { return all + (slot * arrays + array) * size; };
  auto copy = [&](int64_t base, int slot) {
    const int64_t row = base + sub;
    c.copy(place(slot, 0), a.x, a.ld, row, row < a.T);
    c.copy(place(slot, 1), a.dy, a.ld_dy, row, row < a.T);
    if (a.r) c.copy(place(slot, 2), a.r, a.ld_r, row, row < a.T);
    cp_commit();
  };
  for (int i = 0; i < depth; ++i) copy(first + i * step, i);
  float w[EPT], dw[EPT];
  c.weights(a.w, a.w_type, w);
#pragma unroll
  for (int i = 0; i < EPT; ++i) dw[i] = 0.f;
  const float over = 1.f / static_cast<float>(a.D);
  int slot = 0, odd = 0;
#pragma unroll 1
  for (int64_t base = first; base < a.T; base += step) {
    const int64_t row = base + sub;
    const bool on = row < a.T;
    cp_wait(depth - 1);
    Pack<DT, N> ph[V], pd[V], pr[V];
    auto take_dh = [&](int i) {
      if (a.r) c.take(place(slot, 2), i, pr[i]);
      else pr[i].zero();
    };
    auto next = [&] {                               // the slot has been read
      copy(base + depth * step, slot);
      if (++slot == depth) slot = 0;
    };
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c.take(place(slot, 0), i, ph[i]);
      c.take(place(slot, 1), i, pd[i]);
      if constexpr (kEarly) take_dh(i);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float h = ph[i].get(j);
        sum[0] = fmaf(h, h, sum[0]);
        sum[1] = fmaf(pd[i].get(j) * w[i * N + j], h, sum[1]);
      }
    }
    row_sum<2>(sum, threads, part[odd]);
    odd ^= 1;
    if constexpr (kEarly) next();
    // (a row past T, of a block's last step, adds nothing to dw, also where eps is 0)
    const float rstd = on ? 1.f / sqrtf(sum[0] * over + a.eps) : 0.f;
    const float back = rstd * rstd * (sum[1] * over);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (!kKept) {
        c.take(place(slot, 0), i, ph[i]);
        c.take(place(slot, 1), i, pd[i]);
      }
      if constexpr (!kEarly) take_dh(i);
      float f[N];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float h = ph[i].get(j), d = pd[i].get(j);
        f[j] = rstd * fmaf(d, w[i * N + j], -h * back) + pr[i].get(j);
        dw[i * N + j] = fmaf(d, h * rstd, dw[i * N + j]);
      }
      if (on && c.any(i)) {
        Pack<DT, N> p;
        pack<DT, N>(p, f);
        c.put(a.y, row, i, p);
      }
    }
    if constexpr (!kEarly) next();
  }
  cp_wait(0);
  // the block's sums: of its rows side by side, where those are several, in their order; a
  // block alone needs no second launch (one row of 6144 7.0 -> 3.6 us)
  const bool alone = gridDim.x == 1;
  if (alone && rows == 1) {
    const bool vectors = ALIGNED && (reinterpret_cast<uintptr_t>(a.dw) & 15u) == 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!c.any(i)) continue;
      float f[N];
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = dw[i * N + j];
      if (vectors && a.w_type == NVFP4_FP32) {
#pragma unroll
        for (int j = 0; j < N; j += 4)
          *reinterpret_cast<float4*>(static_cast<float*>(a.dw) + c.column(i) + j) =
              make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
      } else if (vectors) {                         // the rows' type
        Pack<DT, N> p;
        pack<DT, N>(p, f);
        c.put(a.dw, 0, i, p);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (c.in(i, j)) put_dw(a.dw, a.w_type, c.column(i) + j, f[j]);
      }
    }
    return;
  }
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * a.D;
  float* all_rows = reinterpret_cast<float*>(staged);            // [rows][D]
  if (rows > 1 || alone) {
    __syncthreads();
    out = all_rows + sub * a.D;
  }
  // (by sixteen bytes: few rows of 6144 7.3 -> 5.3 us, 1000 of them 17 -> 15 us)
  const bool vectors = ALIGNED && (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (vectors) {
      if (c.any(i)) {
#pragma unroll
        for (int j = 0; j < N; j += 4)
          *reinterpret_cast<float4*>(out + c.column(i) + j) =
              make_float4(dw[i * N + j], dw[i * N + j + 1], dw[i * N + j + 2], dw[i * N + j + 3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (c.any(i) && c.in(i, j)) out[c.column(i) + j] = dw[i * N + j];
    }
  }
  if (rows > 1 || alone) {
    __syncthreads();
    for (int col = threadIdx.x; col < a.D; col += blockDim.x) {
      float v = 0.f;
      for (int r = 0; r < rows; ++r) v += all_rows[r * a.D + col];
      if (alone) put_dw(a.dw, a.w_type, col, v);
      else a.part[static_cast<int64_t>(blockIdx.x) * a.D + col] = v;
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
  // launched to overlap the end of the blocks that write the parts
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c < D)
#pragma unroll 8
    for (int p = warp; p < parts; p += 32) v += part[static_cast<int64_t>(p) * D + c];
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < D) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sums[i][lane];
    put_dw(dw, type, c, v);
  }
}

// Elements a thread takes of a row: 8 while there are few rows (a row's time is then
// its latency) or a row has few elements, 16 where rows fill the SMs anyway or 1024 threads
// of 8 are too narrow, 32 for rows that are wider than the threads of 16 that an SM has
// registers for: 768 of 80 (codes with residual of 4096 x 12288 64 us, by 32 elements 96), 512
// of 128.  Registers a thread: 64, `most`, kWideRegs for the grid (up to five warps share the
// 16384 of a quarter of the SM; codes and gradients have up to four, and 128 registers, but for
// the widest gradients begun inside a chunk).
NormShape shape_of(int64_t T, int64_t D, int dtype, int arrays, int most, int rounds,
                   bool aligned) {
  const int es = dtype == NVFP4_FP32 ? 4 : 2;
  const int64_t width = aligned ? D : D + 16 / es - 1;          // begun anywhere in a chunk
  NormShape s{};
  const int widest = (most <= 80 ? 768 : 512) * 16;
  const bool many = T > 2 * kSms && width > 32 * 4 * 8;
  s.ept = width > widest ? 32 : many || width > 1024 * 8 ? 16 : 8;
  s.threads = static_cast<int>((width + 32 * s.ept - 1) / (32 * s.ept)) * 32;
  s.rows = s.threads >= 256 ? 1 : 256 / s.threads;
  const int block = s.threads * s.rows;
  const int regs = s.ept == 8 ? 64 : s.ept == 16 ? most : kWideRegs;
  const int quarter = 16384 / (regs * 32), warps = block / 32;
  int per_sm = quarter / ((warps + 3) / 4);
  // (rows begun anywhere have a warp more: blocks share the quarters unevenly, and two of 13
  // warps with 72 registers fit, 8192 x 6143 59 -> 57 us, 1000 x 6143 10.4 -> 9.3)
  if (!aligned && arrays < kGradArrays) per_sm = quarter * 4 / warps;
  if (per_sm > 2048 / block) per_sm = 2048 / block;
  if (per_sm > 8) per_sm = 8;
  if (per_sm < 1) per_sm = 1;
  // rows on their way: what fits beside the other blocks of the SM
  const int64_t row_bytes = static_cast<int64_t>(block) * s.ept * es * arrays;
  const int64_t want = (T + s.rows - 1) / s.rows;
  while (per_sm > 1 && row_bytes * 2 > kNormSmem / per_sm) --per_sm;
  int64_t depth = kNormSmem / per_sm / row_bytes;
  if (depth > kMostDepth) depth = kMostDepth;
  // (the grid: a multiple of eight, or one step for every block)
  int64_t grid = static_cast<int64_t>(kSms) * per_sm;
  // Many rows: several rounds of blocks, since SMs are not equally fast (norm with residual
  // of 8192 x 6144 72 -> 65 us); not where one block fills an SM (4096 x 8192 47 -> 50 us),
  // nor for the codes.
  if (rounds > 1 && per_sm > 1 && want >= 4 * rounds * grid) grid *= rounds;
  s.grid = static_cast<int>(want < grid ? want : grid);
  const int64_t steps = s.grid > 0 ? (want + s.grid - 1) / s.grid : 1;
  if (depth > steps) depth = steps;
  s.depth = static_cast<int>(depth < 1 ? 1 : depth);
  s.smem = static_cast<size_t>(row_bytes) * s.depth;
  return s;
}
int forward_arrays(const NormArgs& a) { return a.r ? 2 : 1; }

template <int DT, int EPT, bool FP8, bool ALIGNED, int REGS>
cudaError_t go(const NormArgs& a, const NormShape& s, cudaStream_t st) {
  rms_norm_kernel<DT, EPT, FP8, ALIGNED, REGS>
      <<<s.grid, s.threads * s.rows, s.smem, st>>>(a, s.threads, s.rows, s.depth);
  return cudaGetLastError();
}
template <int DT, bool FP8, bool ALIGNED>
cudaError_t forward(const NormArgs& a, int dtype, cudaStream_t st) {
  constexpr int kRegs = FP8 ? kFp8Regs : ALIGNED ? kForwardRegs : kOddRegs;
  const NormShape s = shape_of(a.T, a.D, dtype, forward_arrays(a), kRegs, FP8 ? 1 : 4, ALIGNED);
  if (s.ept == 8) return go<DT, 8, FP8, ALIGNED, 64>(a, s, st);
  if (s.ept == 16) return go<DT, 16, FP8, ALIGNED, kRegs>(a, s, st);
  return go<DT, 32, FP8, ALIGNED, FP8 ? kWideFp8Regs : kWideRegs>(a, s, st);
}

template <int DT, int EPT, bool ALIGNED, int REGS>
void go_grad(const NormArgs& a, const NormShape& s, cudaStream_t st) {
  rms_norm_grad_kernel<DT, EPT, ALIGNED, REGS>
      <<<s.grid, s.threads * s.rows, s.smem, st>>>(a, s.threads, s.rows, s.depth);
}
template <int DT, bool ALIGNED>
cudaError_t backward(const NormArgs& a, int dtype, cudaStream_t st) {
  const NormShape s = shape_of(a.T, a.D, dtype, kGradArrays, kGradRegs, 1, ALIGNED);
  if (s.grid > 0) {
    if (s.ept == 8) go_grad<DT, 8, ALIGNED, 64>(a, s, st);
    else if (s.ept == 16) go_grad<DT, 16, ALIGNED, kGradRegs>(a, s, st);
    else if (ALIGNED || s.threads <= 512) go_grad<DT, 32, ALIGNED, kWideGradRegs>(a, s, st);
    else go_grad<DT, 32, false, kWideRegs>(a, s, st);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || s.grid == 1) return e;
  }
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.D + 31) / 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cfg.attrs = attr;
  attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = s.grid > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, rms_norm_dw_kernel, static_cast<const float*>(a.part), s.grid, a.D,
                            a.w_type, a.dw);
}

template <int DT, int EPT, int REGS, int ODD_REGS, int FP8_REGS, int GRAD_REGS>
cudaError_t set_smem() {
  constexpr auto kAttr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(rms_norm_kernel<DT, EPT, false, true, REGS>, kAttr, kNormSmemMost);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(rms_norm_kernel<DT, EPT, false, false, ODD_REGS>, kAttr, kNormSmemMost);
  if constexpr (DT != NVFP4_FP32)
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(rms_norm_kernel<DT, EPT, true, true, FP8_REGS>, kAttr, kNormSmemMost);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(rms_norm_grad_kernel<DT, EPT, true, GRAD_REGS>, kAttr, kNormSmemMost);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(rms_norm_grad_kernel<DT, EPT, false, GRAD_REGS>, kAttr, kNormSmemMost);
  return e;
}
template <int DT>
cudaError_t set_all() {
  cudaError_t e = set_smem<DT, 8, 64, 64, 64, 64>();
  if (e == cudaSuccess) e = set_smem<DT, 32, kWideRegs, kWideRegs, kWideFp8Regs, kWideGradRegs>();
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(rms_norm_grad_kernel<DT, 32, false, kWideRegs>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmemMost);
  if (e == cudaSuccess) e = set_smem<DT, 16, kForwardRegs, kOddRegs, kFp8Regs, kGradRegs>();
  return e;
}

// Whether every row is made of whole chunks.
bool aligned(const NormArgs& a, int dtype, bool grad) {
  const int es = dtype == NVFP4_FP32 ? 4 : 2;
  auto row16 = [&](const void* p, int64_t ld) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (a.T <= 1 || ld * es % 16 == 0));
  };
  return static_cast<int64_t>(a.D) * es % 16 == 0 && row16(a.x, a.ld) && row16(a.r, a.ld_r) &&
         row16(a.h, a.D) && row16(a.y, a.D) && (!grad || row16(a.dy, a.ld_dy));
}

template <int DT>
cudaError_t by_alignment(const NormArgs& a, int dtype, bool fp8, cudaStream_t st) {
  if constexpr (DT != NVFP4_FP32)
    if (fp8) return forward<DT, true, true>(a, dtype, st);
  return aligned(a, dtype, false) ? forward<DT, false, true>(a, dtype, st)
                                  : forward<DT, false, false>(a, dtype, st);
}
template <int DT>
cudaError_t grad_by_alignment(const NormArgs& a, int dtype, cudaStream_t st) {
  return aligned(a, dtype, true) ? backward<DT, true>(a, dtype, st)
                                 : backward<DT, false>(a, dtype, st);
}

}  // namespace

cudaError_t init_norm_attributes() {
  cudaError_t e = set_all<NVFP4_BF16>();
  if (e == cudaSuccess) e = set_all<NVFP4_FP16>();
  if (e == cudaSuccess) e = set_all<NVFP4_FP32>();
  return e;
}

int norm_grad_parts(int64_t T, int64_t D, int dtype) {
  const int other = shape_of(T, D, dtype, kGradArrays, kGradRegs, 1, false).grid;
  if (D % (dtype == NVFP4_FP32 ? 4 : 8)) return other;
  const int whole = shape_of(T, D, dtype, kGradArrays, kGradRegs, 1, true).grid;
  return whole > other ? whole : other;
}

cudaError_t launch_rms_norm(const NormArgs& a, int dtype, bool fp8, cudaStream_t s) {
  if (dtype == NVFP4_BF16) return by_alignment<NVFP4_BF16>(a, dtype, fp8, s);
  if (dtype == NVFP4_FP16) return by_alignment<NVFP4_FP16>(a, dtype, fp8, s);
  return by_alignment<NVFP4_FP32>(a, dtype, fp8, s);
}

cudaError_t launch_rms_norm_grad(const NormArgs& a, int dtype, cudaStream_t s) {
  if (dtype == NVFP4_BF16) return grad_by_alignment<NVFP4_BF16>(a, dtype, s);
  if (dtype == NVFP4_FP16) return grad_by_alignment<NVFP4_FP16>(a, dtype, s);
  return grad_by_alignment<NVFP4_FP32>(a, dtype, s);
}

}  // namespace nvfp4
