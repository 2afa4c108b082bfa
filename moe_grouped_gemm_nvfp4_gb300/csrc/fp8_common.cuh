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

// The producer's and the MMA's loops run in one lane of their warp, picked once:
// an elect per instruction and a vote per wait made the MMA warp the slowest
// part of the kernel (800 cycles per K block of 256).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 l;\n\t"
      "elect.sync l|e, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r != 0;
}

// D[tmem] = A[smem] . B[smem]^T over one K block: four K = 32 MMAs, 32 bytes
// apart in the 128-byte swizzle.  Columns past K hold zeros.
__device__ __forceinline__ void tc_mma_e4m3_k128(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                 uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred first, rest;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 first, 0, 0;\n\tsetp.ne.b32 rest, 1, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, first;\n\t"
      "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, rest;\n\t"
      "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, rest;\n\t"
      "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, rest;\n\t}"
      :: "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc) : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int32_t x,
                                            int32_t y, int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z),
         "l"(policy)
      : "memory");
}
// Two FP32 values in one 64-bit register, as the packed FMA takes them.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
// acc += {t0, t1} * f.  volatile: not before the wait for the loads of t.
__device__ __forceinline__ void fma_pair(uint64_t& acc, uint32_t t0, uint32_t t1, uint64_t f) {
  asm volatile("{\n\t.reg .b64 t;\n\t"
               "mov.b64 t, {%1, %2};\n\t"
               "fma.rn.f32x2 %0, t, %3, %0;\n\t}"
               : "+l"(acc) : "r"(t0), "r"(t1), "l"(f));
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" :: "r"(addr), "f"(v) : "memory");
}

// Programmatic dependent launch: the GEMM may start while the quantiser before
// it runs; it waits (until that grid has completed and its writes are visible)
// before it touches codes or scales.  Returns at once otherwise.
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One FP32 value as the output type's bits (16-bit types in the low half).
__device__ __forceinline__ uint16_t f32_to_out16(float f, int type) {
  return type == NVFP4_FP16 ? __half_as_ushort(__float2half_rn(f)) : f32_to_bf16_rn(f);
}

// mbar_wait for waits that come once per K block: the clock is read only after
// some tries, since the barrier usually completes within a few hundred cycles
// and reading the global timer takes longer than that.
__device__ __forceinline__ bool wait_soon(uint32_t bar, uint32_t parity, CtaCtl* ctl, int* status) {
  for (int i = 0; i < 32; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, ctl, status);
}

// Two barriers at once: their first tries overlap.
__device__ __forceinline__ bool wait_both(uint32_t bar0, uint32_t parity0, uint32_t bar1,
                                          uint32_t parity1, CtaCtl* ctl, int* status) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "and.pred p, p, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar0), "r"(parity0), "r"(bar1), "r"(parity1) : "memory");
  return ok || (wait_soon(bar0, parity0, ctl, status) && wait_soon(bar1, parity1, ctl, status));
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

// Work units in the order expert, weight tile, token tile: token tiles of one
// weight tile are neighbours, so that all but the first find the weights in L2.
// One matrix: in groups of kTileGroup token tiles, whose activations then stay
// in L2 while the weights pass.
constexpr int kTileGroup = 32;
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
    const int g = u / (kTileGroup * m.ntiles);            // group of token tiles
    const int wide = min(kTileGroup, m.ttiles - g * kTileGroup);
    const int local = u - g * kTileGroup * m.ntiles;
    r.nt = local / wide;
    r.row = (g * kTileGroup + local - r.nt * wide) * m.width;
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
// and the error is recorded.  Offsets that go back and forth would count the same
// rows many times and run over the 32-bit units, so the tiles end where those of
// disjoint experts must (the bound the launcher checks); each stays in its rows.
__device__ __forceinline__ void load_units(const int32_t* offsets, int E, int rows, int width,
                                           int* first, int* tiles, int* status) {
  for (int i = threadIdx.x; i <= E; i += blockDim.x) first[i] = __ldg(offsets + i);
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int some = min(rows, E);
    const int limit = some + (rows - some) / width;
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
      if (e < E) tiles[e] = min(base + incl - n, limit);
      base = min(base + __shfl_sync(0xFFFFFFFFu, incl, 31), limit);
    }
    if (lane == 0) tiles[E] = base;
  }
  __syncthreads();
}

// One warp turns the scales of its units' K blocks [kb0, kb1) into factors in
// shared memory, sa[row] * sw for ROWS tokens, one set per accumulator buffer;
// `put(b, phase)` waits until the buffer is free, `done(b)` tells the epilogue.
// kAhead K blocks' loads are on their way while the group before is written, the
// next unit's first ones behind a unit's last: an L2 read takes longer than a K
// block.  (sa is read by ordinary loads: it may have been written while this
// kernel already ran, which read-only loads rule out.)
constexpr int kAhead = 4;
template <int ROWS, int BUFS, class Put, class Done>
__device__ __forceinline__ void factor_units(const Fp8GemmArgs& a, const UnitMap& um, int u,
                                             int units, int ustep, int kb0, int kb1, uint32_t fac,
                                             int lane, Put put, Done done) {
  constexpr int kPer = (ROWS + 31) / 32;
  if (u >= units) return;
  const float* sw = nullptr;
  const float* sa = nullptr;
  int rows = 0, kb = kb0;
  auto open = [&] {
    const Unit un = unit_at(um, u);
    sw = a.sw + (static_cast<int64_t>(un.e) * a.nnb + un.nt) * a.nkb;
    sa = a.sa + kb0 * a.lds + un.row + lane;
    rows = un.cnt - lane;                        // rows of this lane: 32 * i < rows
    kb = kb0;
  };
  float na[kAhead][kPer], nw[kAhead];
  int nn = 0;                                    // K blocks of the fetched group
  auto fetch = [&] {
    nn = u < units ? min(kAhead, kb1 - kb) : 0;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const bool in = j < nn;
      nw[j] = in ? __ldg(sw + kb + j) : 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) na[j][i] = in && 32 * i < rows ? sa[32 * i] : 0.f;
      sa += a.lds;
    }
    kb += kAhead;
    if (nn > 0 && kb >= kb1) {
      u += ustep;
      if (u < units) open();
    }
  };
  open();
  fetch();
  int buf = 0;
  uint32_t phase = 0;
  while (nn > 0) {
    const int n = nn;
    float f[kAhead][kPer];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int i = 0; i < kPer; ++i) f[j][i] = na[j][i] * nw[j];
    fetch();
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (j >= n) break;
      if (!put(buf, phase)) return;
#pragma unroll
      for (int i = 0; i < kPer; ++i) st_shared_f32(fac + 4 * (buf * 128 + lane + 32 * i), f[j][i]);
      __syncwarp();
      if (lane == 0) done(buf);
      if (++buf == BUFS) { buf = 0; phase ^= 1u; }
    }
  }
}

// n K blocks of one unit added into acc (COLS FP32 values, packed in pairs),
// 32 columns at a time, the next 32 on their way meanwhile.  `wait(b, phase)`
// waits for buffer b's sums and factors (false: give up), `factor(b)` is this
// thread's factor, `release(b)` hands the buffer back; buf and phase run on from
// unit to unit.  False after a wait that gave up.
template <int COLS, int BUFS, class Wait, class Factor, class Release>
__device__ __forceinline__ bool add_unit(uint64_t (&acc)[COLS / 2], int n, uint32_t tbase,
                                         int& buf, uint32_t& phase, Wait wait, Factor factor,
                                         Release release) {
  static_assert(COLS % 64 == 0, "the next block starts at r[0] again");
  uint32_t r[2][32];
  if (!wait(buf, phase)) return false;
  tmem_ld32(tbase + buf * 128, r[0]);
  float f = factor(buf);
  for (int kb = 0; kb < n; ++kb) {
    const uint32_t taddr = tbase + buf * 128;
    const uint64_t ff = pack2(f, f);
#pragma unroll
    for (int c = 0; c < COLS / 32; ++c) {
      tmem_ld_wait();
      if (c + 1 < COLS / 32) {
        tmem_ld32(taddr + 32 * (c + 1), r[(c + 1) & 1]);
      } else {
        release(buf);
        if (++buf == BUFS) { buf = 0; phase ^= 1u; }
        if (kb + 1 < n) {
          if (!wait(buf, phase)) return false;
          tmem_ld32(tbase + buf * 128, r[0]);
          f = factor(buf);
        }
      }
#pragma unroll
      for (int i = 0; i < 32; i += 2)
        fma_pair(acc[(c * 32 + i) / 2], r[c & 1][i], r[c & 1][i + 1], ff);
    }
  }
  return true;
}

// A warp's 32 rows x COLS columns of outputs, row `lane` of them in each lane's
// acc; rows from `rows` on and columns from N on are not stored.  VEC: every row
// is 16-byte aligned and leaves by 16 bytes a lane.  Others (an odd row stride)
// pass through `buf`, 32 rows of 16 words and one of padding, so that a store
// covers 64 bytes of one row: by element from each lane's own row, 9995 routes of
// 1329 columns (K 400) took 127 us, like this 36 us.  (Two kernels: with both ways
// in one the accumulation loop came out 10% slower.)
constexpr int kStoreWords = 32 * 17;
template <int COLS, bool VEC>
__device__ __forceinline__ void store_rows(const Fp8GemmArgs& a, int row0, int rows, int n0,
                                           const uint64_t (&acc2)[COLS / 2], uint32_t buf,
                                           int lane) {
  const int n = a.N - n0;
  if (n <= 0) return;
  float acc[COLS];
#pragma unroll
  for (int i = 0; i < COLS / 2; ++i) unpack2(acc2[i], acc[2 * i], acc[2 * i + 1]);
  const bool wide = a.out_type == NVFP4_FP32;
  if constexpr (VEC) {
    if (lane >= rows) return;
    const int64_t at = static_cast<int64_t>(row0 + lane) * a.ldc + n0;
    if (wide) {
      float* dst = static_cast<float*>(a.out) + at;
#pragma unroll
      for (int i = 0; i < COLS; i += 4) {
        if (i + 4 <= n) {
          *reinterpret_cast<float4*>(dst + i) =
              make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (i + j < n) dst[i + j] = acc[i + j];
        }
      }
    } else {
      uint16_t* dst = static_cast<uint16_t*>(a.out) + at;
#pragma unroll
      for (int i = 0; i < COLS; i += 8) {
        uint16_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = f32_to_out16(acc[i + j], a.out_type);
        if (i + 8 <= n) {
          *reinterpret_cast<uint4*>(dst + i) =
              make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                         h[6] | (h[7] << 16));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (i + j < n) dst[i + j] = h[j];
        }
      }
    }
  } else {
    const int live = min(rows, 32);
    if (wide) {
      float* out = static_cast<float*>(a.out) + static_cast<int64_t>(row0) * a.ldc + n0;
#pragma unroll
      for (int c = 0; c < COLS; c += 16) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) st_shared_f32(buf + 4 * (lane * 17 + i), acc[c + i]);
        __syncwarp();
        const int col = c + (lane & 15);
        for (int r = lane >> 4; r < live; r += 2) {
          const float v = ld_shared_f32(buf + 4 * (r * 17 + (lane & 15)));
          if (col < n) out[r * a.ldc + col] = v;
        }
      }
    } else {
      uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(row0) * a.ldc + n0;
#pragma unroll
      for (int c = 0; c < COLS; c += 32) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          st_shared_f32(buf + 4 * (lane * 17 + i),
                        __uint_as_float(f32_to_out16(acc[c + 2 * i], a.out_type) |
                                        (f32_to_out16(acc[c + 2 * i + 1], a.out_type) << 16)));
        __syncwarp();
        const int col = c + lane;
        for (int r = 0; r < live; ++r) {
          const uint32_t v = __float_as_uint(ld_shared_f32(buf + 4 * (r * 17 + (lane >> 1))));
          if (col < n) out[r * a.ldc + col] = static_cast<uint16_t>(v >> (16 * (lane & 1)));
        }
      }
    }
  }
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
