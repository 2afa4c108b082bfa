// A whole MoE layer for a few tokens (up to 16) over FP8 experts, in one launch:
//
//   l = x . router^T;  experts e_tk and weights w_tk by the top-k gate (gate.cuh)
//   h_tk = SiLU(xq . gate_e^T) * (xq . up_e^T),   out_t = sum_k w_tk hq_tk . down_e^T
//
// with xq and hq the rows' E4M3 codes with 1 x 128 scales (fp8_quant.cuh; h from FP32)
// and FP32 sums in a fixed order: results repeat bit for bit.
//
// Bound: the chosen experts' bytes (HBM).  The design serves that stream:
//
// * One block per SM (a cooperative launch: the blocks meet at two grid barriers, after
//   the router and after h), eight warps, each with a shared-memory ring of its own that
//   it fills by 16-byte asynchronous copies several stages ahead: no barrier inside the
//   stream, and about 100 KB on the way per SM.  At the end of gate_up a warp starts its
//   down copies before it waits for the other blocks, so HBM does not idle there.
// * Work is items of 16 weight rows (8 gate rows and the 8 up rows of the same columns,
//   so that a thread holds both factors of its h; or 16 down rows), expert by expert.  A
//   block takes a contiguous run of items and cuts its K blocks (128 codes of each of the
//   16 rows, 2 KB) into eight equal runs, one a warp.  An item that lies across warps is
//   joined through shared memory in warp order.
// * The tokens are the MMA's 8 columns: m16n8k32 with E4M3 operands, FP32 accumulators
//   cleared every K block and added with both scales.  The matrix pipe idles nearly
//   always (a warp's 2 KB take four instructions), so that the tensor memory path's
//   128-row tiles and set-up would buy nothing here: what counts is that a token's
//   experts divide into two thousand small items instead of hundreds of large ones.
//   Within a K block the order of k is free as long as weights and activations share it:
//   a lane takes 16 consecutive bytes of a row for two MMAs, one 16-byte read each.
// * The down products go out as FP32 rows per route; the last block to finish 16 columns
//   (an arrival counter) adds the routes of each token in order with their weights.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "fp8.h"
#include "fp8_moe.h"
#include "fp8_quant.cuh"

namespace cg = cooperative_groups;

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kItemRows = 16;
constexpr int kStageBytes = kItemRows * 128;
constexpr size_t kMoeSmemMost = (227 - 13) * 1024;     // beside the static arrays

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  const int n = in ? 16 : 0;                            // the rest of the 16 bytes: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// c += A (16 x 32, rows) . B (32 x 8): a0, a2 row g, a1, a3 row g + 8.
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The distinct experts in order of first appearance, and each one's routes.
struct Routes {
  int16_t expert[kMoeMaxRoutes];            // of each route, -1: none
  float weight[kMoeMaxRoutes];
  int16_t live[kMoeMaxRoutes];              // experts' numbers
  int16_t start[kMoeMaxRoutes + 1];         // first of each live expert's entries in `route`
  int16_t route[kMoeMaxRoutes];
  int16_t at[kMoeMaxRoutes];                // start of a leading route's expert
  int n_live;
};

// One phase's matrix and the block's part of its items.
struct Phase {
  const uint8_t* w;
  const float* s;
  int K, nkb, nnb;                          // bytes of a row; blocks of K and of rows
  int units;                                // items of an expert
  int rows;                                 // rows of an expert's matrix
  int half;                                 // gate_up: I; down: 0
  int first, count;                         // the block's items
};

__device__ __forceinline__ int share(int64_t n, int part, int parts) {
  return static_cast<int>(n * part / parts);
}

// Where a warp stands in its run of K blocks.
struct Cursor {
  int left;                                 // K blocks to go
  int x, unit, kb;
  __device__ __forceinline__ void start(const Phase& p, int warp) {
    const int64_t n = static_cast<int64_t>(p.count) * p.nkb;
    const int a = share(n, warp, kWarps), b = share(n, warp + 1, kWarps);
    left = b - a;
    const int item = p.first + a / p.nkb;
    kb = a % p.nkb;
    x = item / p.units;
    unit = item - x * p.units;
  }
  __device__ __forceinline__ void next(const Phase& p) {
    --left;
    if (++kb == p.nkb) {
      kb = 0;
      if (++unit == p.units) { unit = 0; ++x; }
    }
  }
};

// Copies of one K block of 16 rows into a stage: instruction i takes rows 4 i to 4 i + 3,
// eight lanes a row.  In shared memory the 16-byte chunks of odd rows lie 64 bytes on
// (modulo 128), so that two rows' reads of four chunks fall into different banks.
__device__ __forceinline__ void fetch(const Phase& p, const Routes& rt, const Cursor& c,
                                      uint32_t stage, uint32_t scales) {
  const int lane = threadIdx.x & 31;
  const int e = rt.live[c.x];
  const int chunk = lane & 7;
  const int k = c.kb * 128 + chunk * 16;
  const bool in = k < p.K;
  const int r0 = lane >> 3;
  // rows of the unit: 8 of each half (gate, up), or 16 of the matrix
  const int base = p.half ? c.unit * 8 : c.unit * 16;
  const int64_t first = static_cast<int64_t>(e) * p.rows;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * i + r0;
    int row = base + r;
    if (p.half) row = i < 2 ? row : p.half + row - 8;
    else row = min(row, p.rows - 1);
    const uint8_t* src = p.w + (first + row) * p.K + (in ? k : 0);
    cp16(stage + r * 128 + ((chunk ^ ((r & 1) << 2)) << 4), src, in);
  }
  if (lane < 2) {
    const int row = lane && p.half ? p.half + base : base;
    cp4(scales + lane * 4,
        p.s + (static_cast<int64_t>(e) * p.nnb + row / kFp8Block) * p.nkb + c.kb);
  }
}

// Rows of activations as E4M3 codes in shared memory: row r at r * stride, chunks of 16
// in order; the scales of its K blocks.
struct Acts {
  uint32_t codes;
  int stride;
  float* scale;                             // [rows][nkb]
  int nkb;
};

template <class Scale>
__device__ __forceinline__ void put_codes(const Acts& s, int row, int k, const float (&v)[16]) {
  const Scale b(block_amax(v));
  if (k >= s.nkb * 128) return;
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    q[j] = e4m3x4(b.quotient(v[4 * j]), b.quotient(v[4 * j + 1]), b.quotient(v[4 * j + 2]),
                  b.quotient(v[4 * j + 3]));
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(s.codes + row * s.stride + k),
               "r"(q[0]), "r"(q[1]), "r"(q[2]), "r"(q[3]) : "memory");
  if ((threadIdx.x & 7) == 0) s.scale[row * s.nkb + k / kFp8Block] = b.scale;
}

// An item that a warp's run of K blocks begins and does not end.
struct Tail {
  int x, unit;                              // x < 0: none
};

template <int DT, int NT, int S>
struct Layer {
  const Fp8MoeArgs& a;
  const Routes& rt;
  float (*head)[32][NT * 4];                // sums of items that an earlier warp began
  uint32_t ring, ring_scale;                // of this warp
  int warp, lane;

  __device__ __forceinline__ uint32_t stage(int i) const { return ring + i * kStageBytes; }
  __device__ __forceinline__ uint32_t scales(int i) const { return ring_scale + i * 8; }

  // The first S - 1 stages on their way.
  __device__ __forceinline__ void prime(const Phase& p, Cursor& in) const {
    __syncwarp();
    in.start(p, warp);
#pragma unroll 1
    for (int i = 0; i < S - 1; ++i) {
      if (in.left > 0) {
        fetch(p, rt, in, stage(i), scales(i));
        in.next(p);
      }
      cp_commit();
    }
  }

  // A finished item: h of the expert's routes, or their rows of the output.
  template <bool DOWN>
  __device__ __forceinline__ void finish(int x, int unit, const float (&acc)[NT][4]) const {
    const int first = rt.start[x], n = rt.start[x + 1] - first;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = nt * 8 + 2 * t + i;
        if (j >= n) continue;
        const int64_t r = rt.route[first + j];
        if constexpr (DOWN) {
          const int c = unit * 16 + g;
          if (c < a.N) __stcg(a.part + r * a.N + c, acc[nt][i]);
          if (c + 8 < a.N) __stcg(a.part + r * a.N + c + 8, acc[nt][2 + i]);
        } else {
          const float gate = acc[nt][i], up = acc[nt][2 + i];
          __stcg(a.h + r * a.I + unit * 8 + g, gate / (1.f + __expf(-gate)) * up);
        }
      }
    if constexpr (DOWN) {
      __threadfence();
      __syncwarp();
      uint32_t before = 0;
      if (lane == 0) before = atomicAdd(a.arrived + unit, 1u);
      before = __shfl_sync(kFullWarp, before, 0);
      if (before + 1 != static_cast<uint32_t>(rt.n_live)) return;
      __threadfence();
      for (int i = lane; i < a.T * 16; i += 32) {
        const int tok = i >> 4, c = unit * 16 + (i & 15);
        if (c >= a.N) continue;
        float v = 0.f;
        for (int k = 0; k < a.rule.topk; ++k) {
          const int r = tok * a.rule.topk + k;
          if (rt.expert[r] >= 0)
            v = fmaf(rt.weight[r], __ldcg(a.part + static_cast<int64_t>(r) * a.N + c), v);
        }
        static_cast<uint16_t*>(a.out)[tok * a.ldo + c] = static_cast<uint16_t>(f32_to_elem<DT>(v));
      }
    }
  }

  // The warp's run of K blocks, primed before.  Row of the activations of an entry:
  // its token (gate_up), or its place among the block's entries from entry0 on (down).
  template <bool DOWN>
  __device__ __forceinline__ Tail stream(const Phase& p, const Acts& act, int entry0, Cursor& in,
                                         float (&acc)[NT][4]) const {
    auto act_row = [&](int entry) {
      return DOWN ? entry - entry0 : rt.route[entry] / a.rule.topk;
    };
    Cursor c;
    c.start(p, warp);
    const int g = lane >> 2, t = lane & 3;
    bool is_head = c.left > 0 && c.kb != 0;             // begun by an earlier warp
    uint32_t row[NT];
    int col[NT][2];
    int x = -1, tiles = 0, slot = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      row[nt] = 0;
      col[nt][0] = col[nt][1] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
    }
    while (c.left > 0) {
      cp_wait<S - 2>();
      __syncwarp();                      // the stage is there for every lane, and the one
      if (in.left > 0) {                 // before it has been read by every lane
        const int s = slot == 0 ? S - 1 : slot - 1;
        fetch(p, rt, in, stage(s), scales(s));
        in.next(p);
      }
      cp_commit();
      if (c.x != x) {
        x = c.x;
        const int first = rt.start[x], n = rt.start[x + 1] - first;
        tiles = (n + 7) >> 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // columns past the expert's routes repeat its last one; nobody reads them
          row[nt] = act.codes + act.stride * act_row(first + min(nt * 8 + g, n - 1));
#pragma unroll
          for (int i = 0; i < 2; ++i)
            col[nt][i] = act_row(first + min(nt * 8 + 2 * t + i, n - 1)) * act.nkb;
        }
      }
      const uint32_t st = stage(slot);
      float sum[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[nt][i] = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int chunk = (t + 4 * j) ^ ((g & 1) << 2);
        const uint4 lo = lds128(st + g * 128 + chunk * 16);
        const uint4 hi = lds128(st + (g + 8) * 128 + chunk * 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (nt < tiles) {
            const uint4 b = lds128(row[nt] + c.kb * 128 + (t + 4 * j) * 16);
            mma_e4m3(sum[nt], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
            mma_e4m3(sum[nt], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
          }
        }
      }
      float s_lo, s_hi;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(s_lo), "=f"(s_hi) : "r"(scales(slot))
                   : "memory");
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (nt < tiles) {
          const float a0 = act.scale[col[nt][0] + c.kb], a1 = act.scale[col[nt][1] + c.kb];
          acc[nt][0] = fmaf(sum[nt][0], a0 * s_lo, acc[nt][0]);
          acc[nt][1] = fmaf(sum[nt][1], a1 * s_lo, acc[nt][1]);
          acc[nt][2] = fmaf(sum[nt][2], a0 * s_hi, acc[nt][2]);
          acc[nt][3] = fmaf(sum[nt][3], a1 * s_hi, acc[nt][3]);
        }
      }
      slot = slot + 1 == S ? 0 : slot + 1;
      const int unit = c.unit;
      const bool ends = c.kb == p.nkb - 1;
      c.next(p);
      if (ends || c.left == 0) {
        if (is_head) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) head[warp][lane][nt * 4 + i] = acc[nt][i];
          is_head = false;
        } else if (ends) {
          finish<DOWN>(x, unit, acc);
        } else {
          return Tail{x, unit};
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
      }
    }
    return Tail{-1, 0};
  }

  // After a block barrier: the later warps' sums of the item that this warp began.
  template <bool DOWN>
  __device__ __forceinline__ void join(const Phase& p, const Tail& tail, float (&acc)[NT][4]) const {
    if (tail.x < 0) return;
    const int64_t n = static_cast<int64_t>(p.count) * p.nkb;
    const int end = (tail.x * p.units + tail.unit - p.first + 1) * p.nkb;
    for (int w = warp + 1; w < kWarps; ++w) {
      const int from = share(n, w, kWarps);
      if (from >= end) break;
      if (from == share(n, w + 1, kWarps)) continue;    // no K block of its own
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] += head[w][lane][nt * 4 + i];
    }
    finish<DOWN>(tail.x, tail.unit, acc);
  }
};

// Logits of the block's experts: the warps share K, every one for all tokens.
template <int DT, int RT, int MT>
__device__ __noinline__ void router_logits(const Fp8MoeArgs& a, float (*part)[MT]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int N = elems_per_16b<DT>();
  for (int e = blockIdx.x; e < a.rule.E; e += gridDim.x) {
    float acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = 0.f;
    for (int k = (warp * 32 + lane) * N; k < a.K; k += kThreads * N) {
      float w[N];
      if constexpr (RT == NVFP4_FP32) {
        Pack<NVFP4_FP32, 4> lo, hi;
        lo.load(a.router, static_cast<int64_t>(e) * a.K + k);
        hi.load(a.router, static_cast<int64_t>(e) * a.K + k + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) { w[i] = lo.get(i); w[4 + i] = hi.get(i); }
      } else {
        Pack<RT, N> v;
        v.load(a.router, static_cast<int64_t>(e) * a.K + k);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = v.get(i);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (t < a.T) {
          Pack<DT, N> v;
          v.load(a.x, t * a.ld + k);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[t] = fmaf(v.get(i), w[i], acc[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      acc[t] = warp_sum(acc[t]);
      if (lane == 0) part[warp][t] = acc[t];
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < a.T) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += part[w][threadIdx.x];
      __stcg(a.logits + static_cast<int64_t>(threadIdx.x) * a.rule.E + e, v);
    }
    __syncthreads();
  }
}

template <int L>
__device__ __noinline__ void gate_token(const Fp8MoeArgs& a, Routes& rt, int t) {
  const int lane = threadIdx.x & 31;
  float l[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < a.rule.E ? __ldcg(a.logits + static_cast<int64_t>(t) * a.rule.E + e) : -INFINITY;
  }
  int id;
  float w;
  gate_choose<L>(a.rule, l, &id, &w);
  if (lane < a.rule.topk) {
    const int r = t * a.rule.topk + lane;
    rt.expert[r] = static_cast<int16_t>(id);
    rt.weight[r] = w;
    if (blockIdx.x == 0) {
      a.ids[r] = id;
      a.weights[r] = w;
    }
  }
}

// The routes by expert, the same in every block.
__device__ __noinline__ void list_experts(const Fp8MoeArgs& a, Routes& rt, int2* scan) {
  const int R = a.T * a.rule.topk;
  const int r = threadIdx.x, warp = r >> 5, lane = r & 31;
  if (!a.router && r < a.T) {
    // an expert that a token names twice: once, with both weights
    for (int k = 1; k < a.rule.topk; ++k)
      for (int j = 0; j < k; ++j) {
        const int i = r * a.rule.topk;
        if (rt.expert[i + k] >= 0 && rt.expert[i + k] == rt.expert[i + j]) {
          rt.weight[i + j] += rt.weight[i + k];
          rt.expert[i + k] = -1;
        }
      }
  }
  __syncthreads();
  const int e = r < R ? rt.expert[r] : -1;
  int first = r, place = 0, count = 0;
  if (e >= 0) {
    for (int i = 0; i < R; ++i)
      if (rt.expert[i] == e) {
        first = min(first, i);
        place += i < r;
        ++count;
      }
  }
  const bool lead = e >= 0 && first == r;
  // exclusive sums over the leading routes: experts (x) and entries (y)
  int2 v = make_int2(lead ? 1 : 0, lead ? count : 0);
  const int2 own = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFullWarp, v.x, o), y = __shfl_up_sync(kFullWarp, v.y, o);
    if (lane >= o) { v.x += x; v.y += y; }
  }
  if (lane == 31) scan[warp] = v;
  __syncthreads();
  int2 base = make_int2(v.x - own.x, v.y - own.y);
  for (int w = 0; w < warp; ++w) { base.x += scan[w].x; base.y += scan[w].y; }
  if (lead) {
    rt.live[base.x] = static_cast<int16_t>(e);
    rt.start[base.x] = static_cast<int16_t>(base.y);
    rt.at[r] = static_cast<int16_t>(base.y);
  }
  if (r == kThreads - 1) {
    rt.n_live = base.x + own.x;
    rt.start[base.x + own.x] = static_cast<int16_t>(base.y + own.y);
  }
  __syncthreads();
  if (e >= 0) rt.route[rt.at[first] + place] = static_cast<int16_t>(r);
  __syncthreads();
}

template <int DT, int NT, int S>
__global__ void __launch_bounds__(kThreads, 1) fp8_moe_kernel(const Fp8MoeArgs a,
                                                              const Fp8MoePlan plan) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Routes rt;
  __shared__ float head[kWarps][32][NT * 4];
  __shared__ float part[kWarps][NT * 8];
  __shared__ int2 scan[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem);
  const uint32_t ring_scales = base + kWarps * S * kStageBytes;
  const uint32_t act_codes = ring_scales + kWarps * S * 8;
  float* act_scales = reinterpret_cast<float*>(smem + kWarps * S * (kStageBytes + 8) +
                                               plan.act_rows * plan.act_stride);
  const Layer<DT, NT, S> layer{a, rt, head, base + warp * S * kStageBytes,
                               ring_scales + warp * S * 8, warp, lane};
  cg::grid_group grid = cg::this_grid();

  const int units2 = (a.N + 15) / 16;
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < units2; i += gridDim.x * kThreads)
    __stcg(a.arrived + i, 0u);
  if (a.router) {
    if (a.router_type == NVFP4_FP32) router_logits<DT, NVFP4_FP32, NT * 8>(a, part);
    else router_logits<DT, DT, NT * 8>(a, part);
  }
  Acts act{act_codes, plan.act_stride, act_scales, (a.K + 127) / 128};
  {
    const int chunks = (a.K + 511) / 512;
    for (int i = warp; i < a.T * chunks; i += kWarps) {
      const int t = i / chunks, k = (i - t * chunks) * 512 + lane * 16;
      float v[16];
      if (k < a.K) {
        load_row16<DT, false>(a.x, t * a.ld, a.K, k, v);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0.f;
      }
      put_codes<BlockScale>(act, t, k, v);
    }
  }
  if (a.router) {
    grid.sync();
    for (int t = warp; t < a.T; t += kWarps) {
      if (a.rule.E <= 128) gate_token<4>(a, rt, t);
      else if (a.rule.E <= 256) gate_token<8>(a, rt, t);
      else gate_token<32>(a, rt, t);
    }
  } else {
    const int r = threadIdx.x;
    if (r < a.T * a.rule.topk) {
      const int e = __ldg(a.ids + r);
      const bool ok = e >= 0 && e < a.rule.E;
      if (!ok) raise_status(a.status, NVFP4_ERR_DEVICE_CHECK);
      rt.expert[r] = static_cast<int16_t>(ok ? e : -1);
      rt.weight[r] = __ldg(a.weights + r);
    }
  }
  __syncthreads();
  list_experts(a, rt, scan);

  Phase p;
  auto place = [&](int units) {
    p.units = units;
    const int64_t items = static_cast<int64_t>(rt.n_live) * units;
    p.first = share(items, blockIdx.x, gridDim.x);
    p.count = share(items, blockIdx.x + 1, gridDim.x) - p.first;
  };
  float acc[NT][4];
  Cursor in;
  p.w = a.w1; p.s = a.s1; p.K = a.K; p.nkb = (a.K + 127) / 128;
  p.nnb = (2 * a.I + 127) / 128; p.rows = 2 * a.I; p.half = a.I;
  place(a.I / 8);
  layer.prime(p, in);
  Tail tail = layer.template stream<false>(p, act, 0, in, acc);
  const Phase gate_up = p;
  p.w = a.w2; p.s = a.s2; p.K = a.I; p.nkb = (a.I + 127) / 128;
  p.nnb = (a.N + 127) / 128; p.rows = a.N; p.half = 0;
  place(units2);
  layer.prime(p, in);                       // on their way across the barrier
  __syncthreads();
  layer.template join<false>(gate_up, tail, acc);
  grid.sync();

  act.nkb = (a.I + 127) / 128;
  int entry0 = 0;
  if (p.count > 0) {
    const int x1 = (p.first + p.count - 1) / p.units;
    entry0 = rt.start[p.first / p.units];
    const int rows = rt.start[x1 + 1] - entry0;
    const int chunks = (a.I + 511) / 512;
    for (int i = warp; i < rows * chunks; i += kWarps) {
      const int j = i / chunks, k = (i - j * chunks) * 512 + lane * 16;
      float v[16];
      const float4* src = reinterpret_cast<const float4*>(
          a.h + static_cast<int64_t>(rt.route[entry0 + j]) * a.I + k);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 f = k < a.I ? __ldcg(src + q) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
      }
      put_codes<BlockScale32>(act, j, k, v);
    }
  }
  __syncthreads();
  tail = layer.template stream<true>(p, act, entry0, in, acc);
  __syncthreads();
  layer.template join<true>(p, tail, acc);
  cp_wait<0>();
  if (rt.n_live == 0)                       // no route at all
    for (int64_t i = blockIdx.x * kThreads + threadIdx.x; i < static_cast<int64_t>(a.T) * a.N;
         i += static_cast<int64_t>(gridDim.x) * kThreads)
      static_cast<uint16_t*>(a.out)[i / a.N * a.ldo + i % a.N] = 0;
}

template <int DT, int NT, int S>
cudaError_t go(const Fp8MoeArgs& a, const Fp8MoePlan& p, cudaStream_t s) {
  void* args[] = {const_cast<Fp8MoeArgs*>(&a), const_cast<Fp8MoePlan*>(&p)};
  return cudaLaunchCooperativeKernel(fp8_moe_kernel<DT, NT, S>, dim3(p.grid), dim3(kThreads), args,
                                     p.smem, s);
}
template <int DT, int NT>
cudaError_t by_stages(const Fp8MoeArgs& a, const Fp8MoePlan& p, cudaStream_t s) {
  if (p.stages == 12) return go<DT, NT, 12>(a, p, s);
  if (p.stages == 8) return go<DT, NT, 8>(a, p, s);
  return go<DT, NT, 5>(a, p, s);
}
template <int DT>
cudaError_t by_tiles(const Fp8MoeArgs& a, const Fp8MoePlan& p, cudaStream_t s) {
  return p.tiles == 1 ? by_stages<DT, 1>(a, p, s) : by_stages<DT, 2>(a, p, s);
}

template <int DT, int NT, int S>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(fp8_moe_kernel<DT, NT, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kMoeSmemMost));
}
template <int DT, int NT>
cudaError_t set_stages() {
  cudaError_t e = set_smem<DT, NT, 12>();
  if (e == cudaSuccess) e = set_smem<DT, NT, 8>();
  if (e == cudaSuccess) e = set_smem<DT, NT, 5>();
  return e;
}

}  // namespace

cudaError_t init_fp8_moe_attributes() {
  cudaError_t e = set_stages<NVFP4_BF16, 1>();
  if (e == cudaSuccess) e = set_stages<NVFP4_BF16, 2>();
  if (e == cudaSuccess) e = set_stages<NVFP4_FP16, 1>();
  if (e == cudaSuccess) e = set_stages<NVFP4_FP16, 2>();
  return e;
}

bool fp8_moe_plan(int T, int topk, int E, int64_t K, int64_t I, int64_t N, int sms, Fp8MoePlan* p) {
  if (T > kMoeMaxTokens || T * topk > kMoeMaxRoutes || E > kGateMaxExperts ||
      topk > kGateMaxTopk || K > (1 << 20) || I > (1 << 20) || N > (1 << 20))
    return false;
  p->tiles = T > 8 ? 2 : 1;
  p->grid = sms;
  // the rows of h that a block can need: those of the experts that its items span
  const int64_t R = static_cast<int64_t>(T) * topk, live = R < E ? R : E;
  const int64_t units = (N + 15) / 16, run = (live * units + sms - 1) / sms;
  const int64_t span = run <= 1 ? 1 : (run - 2) / units + 2;
  const int64_t rows = span * T < R ? span * T : R;
  const int64_t kx = (K + 127) / 128, kh = (I + 127) / 128;
  const int64_t wide = kx > kh ? kx : kh;
  p->act_rows = static_cast<int>(T > rows ? T : rows);
  p->act_stride = static_cast<int>(wide * 128 + 64);       // two rows' chunks in different banks
  const int64_t acts = p->act_rows * (p->act_stride + wide * 4);
  for (int s : {12, 8, 5}) {
    const int64_t bytes = static_cast<int64_t>(kWarps) * s * (kStageBytes + 8) + acts;
    if (bytes <= static_cast<int64_t>(kMoeSmemMost)) {
      p->stages = s;
      p->smem = static_cast<size_t>(bytes);
      return true;
    }
  }
  return false;
}

cudaError_t launch_fp8_moe(const Fp8MoeArgs& a, const Fp8MoePlan& p, int dtype, cudaStream_t s) {
  return dtype == NVFP4_BF16 ? by_tiles<NVFP4_BF16>(a, p, s) : by_tiles<NVFP4_FP16>(a, p, s);
}

}  // namespace nvfp4
