// A whole MoE layer for a few tokens (up to 32) over FP8 experts, in one launch:
//
//   l = x . router^T;  experts e_tk and weights w_tk by the top-k gate (gate.cuh)
//   h_tk = SiLU(xq . gate_e^T) * (xq . up_e^T),   out_t = sum_k w_tk hq_tk . down_e^T
//
// with xq and hq the rows' E4M3 codes with 1 x 128 scales (fp8_quant.cuh; h from FP32)
// and FP32 sums in a fixed order: results repeat bit for bit.
//
// Bound: the chosen experts' bytes (HBM).  The design serves that stream:
//
// * One block per SM (a cooperative launch).  The blocks meet at two grid barriers: when
//   the logits and the codes of x are written, and when the codes of h are.
// * Weights are the MMA's 128 rows (tcgen05, M 128), the tokens its 16 or 32 columns: all
//   tokens, so that nothing is gathered; an expert's columns of other tokens are dropped.
//   A tile is 256 weight rows x 128 K (32 KB, two TMA boxes): the gate and up rows of 128
//   columns of h, so that one thread holds both factors of its h, or 256 down rows.
//   Rows past a matrix read as zeros.
// * The tiles of a phase stand in one line (gate_up: expert, 128 columns, K block; down:
//   256 columns, expert, K block) that is cut into equal runs, one a block, wherever that
//   falls: a token's eight experts have some thousands of tiles, and every SM streams the
//   same bytes.  An item (128 columns of one expert's h; 256 output columns over all
//   experts) whose tiles lie in several blocks is joined by the last of them to finish,
//   which adds the parts in block order.
// * Six stages are on their way (192 KB an SM).  When a block has asked for all its gate_up
//   tiles, its producer goes on with the weights of its first down tiles, before the grid
//   barrier that the codes of h wait for: HBM does not idle there.
// * Both scales differ by K block, so every K block has accumulators of its own in tensor
//   memory, which four warps read and add as FP32 times the factor (weight scale * token
//   scale, for down also * routing weight) that a warp of its own lays out.
//
// (A first form with mma.sync, eight warps with rings of their own: it spent 280
// instructions on 2 KB of weights, converting codes, and reached 4.3 TB/s: one token
// through 128 experts of 6144 x 2048, eight of them chosen, in 96 us.)
#include <cooperative_groups.h>

#include "fp8_common.cuh"
#include "fp8_moe.h"
#include "fp8_quant.cuh"

namespace cg = cooperative_groups;

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroupBytes = 128 * 128;      // 128 weight rows of a K block
constexpr int kAccBufs = 8;                 // of 2 x 16 or 2 x 32 columns

// TB: token columns (8, 16 or 32).
template <int TB>
struct Shape {
  static constexpr int kCols = TB < 16 ? 16 : TB;           // of the MMA
  static constexpr int kStages = TB == 32 ? 5 : 6;
  static constexpr int kTokOffset = 2 * kGroupBytes;
  static constexpr int kStageBytes = kTokOffset + kCols * 128;
  static constexpr int kFacOffset = kStages * kStageBytes;  // [bufs][3][TB] floats
  static constexpr int kRedOffset = kFacOffset + kAccBufs * 3 * TB * 4;   // [4][TB] maxima
  static constexpr int kBarOffset = kRedOffset + 4 * TB * 4;
  static constexpr int kCtlOffset = kBarOffset + 8 * (2 * kStages + 2 * kAccBufs + 2);
  static constexpr int kSmemBytes = kCtlOffset + 32 + 1024;
  static constexpr uint32_t kTmemCols = kAccBufs * 2 * kCols;             // 256 or 512
};

// The distinct experts in order of first appearance, and each one's routes.
struct Routes {
  float weight[kMoeMaxRoutes];              // of each route
  uint32_t tokens[kMoeMaxRoutes];           // of each live expert, one bit each
  int16_t expert[kMoeMaxRoutes];            // of each route, -1: none
  int16_t live[kMoeMaxRoutes];              // experts' numbers
  int16_t start[kMoeMaxRoutes];             // first of each live expert's entries in `route`
  int16_t route[kMoeMaxRoutes];
  int n_live;
};

__device__ __forceinline__ void fence_proxy_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// Uses of r stay behind the wait for its load (volatile statements keep their order).
__device__ __forceinline__ void keep_after(uint32_t (&r)[8]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                    "+r"(r[6]), "+r"(r[7]));
}

// One phase's line of tiles and the block's run of it.
struct Phase {
  int down;
  int nkb;                                  // K blocks of an item's expert
  int units;                                // gate_up: ceil(I / 128); down: ceil(N / 256)
  int experts;
  int per_item;                             // tiles of an item
  int grain, grains;                        // runs begin at multiples of `grain` tiles
  int parts;                                // blocks that have tiles
  int first, count;                         // the block's run

  __device__ __forceinline__ int begin(int block) const {
    return grain * static_cast<int>(static_cast<int64_t>(grains) * block / parts);
  }
  // The block whose run holds a tile.
  __device__ __forceinline__ int owner(int tile) const {
    return static_cast<int>(((static_cast<int64_t>(tile / grain) + 1) * parts - 1) / grains);
  }
  // Runs of whole items need no join, which takes about 4 us behind the last tile; runs of
  // single tiles are all equally long.  A tile takes 0.76 us while all SMs draw on HBM and
  // at least 0.53 us (62 GB/s is all that one SM draws); a join 5 tiles' time.  At most about
  // eight blocks share an item: the last one reads all parts.
  __device__ __forceinline__ void set(int is_down, int k_blocks, int n_units, int n_experts) {
    const int blocks = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
    down = is_down;
    nkb = k_blocks;
    units = n_units;
    experts = n_experts;
    per_item = max(down ? nkb * experts : nkb, 1);
    const int items = down ? units * min(experts, 1) : units * experts;
    const int rest = items % blocks;
    const int64_t rounds = 100 * (items / blocks) + (rest ? max(70, 100 * rest / blocks) : 0);
    const bool whole = rounds * per_item <= 100 * static_cast<int64_t>(items) * per_item / blocks + 500;
    grain = whole ? per_item : 1;
    grains = whole ? items : items * per_item;
    parts = min(blocks, min(grains, 8 * items));
    first = b < parts ? begin(b) : 0;
    count = b < parts ? begin(b + 1) - first : 0;
  }
};

// A tile of the line: live expert, unit, K block.
struct Cursor {
  int x, unit, kb;
  __device__ __forceinline__ void at(const Phase& p, int tile) {
    kb = tile % p.nkb;
    const int rest = tile / p.nkb;
    if (p.down) {
      x = rest % max(p.experts, 1);
      unit = rest / max(p.experts, 1);
    } else {
      unit = rest % p.units;
      x = rest / p.units;
    }
  }
  __device__ __forceinline__ void next(const Phase& p) {
    if (++kb < p.nkb) return;
    kb = 0;
    if (p.down) {
      if (++x == p.experts) { x = 0; ++unit; }
    } else {
      if (++unit == p.units) { unit = 0; ++x; }
    }
  }
};

// Shared memory of a block.
template <int TB>
struct Block {
  using S = Shape<TB>;
  uint32_t base;
  uint8_t* smem;
  CtaCtl* ctl;
  int* status;
  uint32_t tmem;
  __device__ __forceinline__ uint32_t stage(int s) const { return base + s * S::kStageBytes; }
  __device__ __forceinline__ uint32_t bar(int i) const { return base + S::kBarOffset + 8u * i; }
  __device__ __forceinline__ uint32_t full(int s) const { return bar(s); }
  __device__ __forceinline__ uint32_t empty(int s) const { return bar(S::kStages + s); }
  __device__ __forceinline__ uint32_t accf(int b) const { return bar(2 * S::kStages + b); }
  __device__ __forceinline__ uint32_t acce(int b) const {
    return bar(2 * S::kStages + kAccBufs + b);
  }
  __device__ __forceinline__ uint32_t drain() const { return bar(2 * S::kStages + 2 * kAccBufs); }
  __device__ __forceinline__ uint32_t meet() const {
    return bar(2 * S::kStages + 2 * kAccBufs + 1);
  }
  __device__ __forceinline__ float* fac(int b) const {
    return reinterpret_cast<float*>(smem + S::kFacOffset) + b * 3 * TB;
  }
  __device__ __forceinline__ float* red() const {
    return reinterpret_cast<float*>(smem + S::kRedOffset);
  }
};

// Counts a role's passes over a ring of n slots.
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) { slot = 0; phase ^= 1u; }
  }
};

// ------------------------------------------------------------------ producer

template <int TB>
struct Producer {
  const Block<TB>& b;
  const Routes& rt;
  const CUtensorMap* w;
  const CUtensorMap* tok;
  uint64_t wpol, tpol;

  __device__ __forceinline__ void weights(const Phase& p, const Cursor& c, int s) const {
    using S = Shape<TB>;
    const int e = rt.live[c.x];
    mbar_arrive_expect_tx(b.full(s), S::kStageBytes);
    if (p.down) {
      tma_load_3d(b.stage(s), w, b.full(s), c.kb * 128, c.unit * 256, e, wpol);
      tma_load_3d(b.stage(s) + kGroupBytes, w, b.full(s), c.kb * 128, c.unit * 256 + 128, e, wpol);
    } else {
      tma_load_3d(b.stage(s), w, b.full(s), c.kb * 128, c.unit * 128, 2 * e, wpol);
      tma_load_3d(b.stage(s) + kGroupBytes, w, b.full(s), c.kb * 128, c.unit * 128, 2 * e + 1,
                  wpol);
    }
  }
  __device__ __forceinline__ void tokens(const Phase& p, const Cursor& c, int s) const {
    tma_load_2d(b.stage(s) + Shape<TB>::kTokOffset, tok, b.full(s), c.kb * 128,
                p.down ? c.x * TB : 0, tpol);
  }
};

// ------------------------------------------------------------------- factors

// One warp: for each tile the products of the weight scales (gate or first 128 rows; up
// or second 128 rows, whose scale can change within the 128 rows where I is no multiple
// of 128) and of each token's scale (times its routing weight in the down phase).
template <int TB>
__device__ __forceinline__ void factors(const Block<TB>& b, const Fp8MoeArgs& a, const Routes& rt,
                                        const Phase& p, Ring& acc) {
  const int lane = threadIdx.x & 31;
  Cursor c;
  c.at(p, p.first);
  const float* ws = p.down ? a.s2 : a.s1;
  const int nnb = p.down ? (a.N + 127) / 128 : (2 * a.I + 127) / 128;
  int x = -1;
  float weight = 1.f;
  struct Raw {
    float tok, w0, w1, w2;
  };
  auto load = [&](const Cursor& at) {
    Raw r;
    const int e = rt.live[at.x];
    const int r0 = p.down ? 2 * at.unit : at.unit;
    const int up = a.I + at.unit * 128;
    const int r1 = p.down ? min(r0 + 1, nnb - 1) : up / 128;
    const int r2 = p.down ? r1 : min(r1 + 1, nnb - 1);
    const float* row = ws + static_cast<int64_t>(e) * nnb * p.nkb + at.kb;
    r.w0 = __ldg(row + static_cast<int64_t>(r0) * p.nkb);
    r.w1 = __ldg(row + static_cast<int64_t>(r1) * p.nkb);
    r.w2 = __ldg(row + static_cast<int64_t>(r2) * p.nkb);
    const float* ts = p.down ? a.hs + (static_cast<int64_t>(at.x) * p.nkb + at.kb) * TB
                             : a.xs + at.kb * TB;
    r.tok = lane < TB && lane < a.T ? __ldcg(ts + lane) : 0.f;
    return r;
  };
  Raw next{};
  if (p.count > 0) next = load(c);
  for (int i = 0; i < p.count; ++i) {
    const Raw r = next;
    if (p.down && c.x != x) {
      x = c.x;
      const uint32_t tokens = rt.tokens[x];
      const int j = rt.start[x] + __popc(tokens & ((1u << lane) - 1u));
      weight = tokens >> lane & 1u ? rt.weight[rt.route[j]] : 0.f;
    }
    c.next(p);
    if (i + 1 < p.count) next = load(c);
    if (!__all_sync(kFullWarp, wait_soon(b.acce(acc.slot), acc.phase ^ 1u, b.ctl, b.status))) return;
    if (lane < TB) {
      float* f = b.fac(acc.slot);
      // the weight's scale first: the product with the token's stays in the result's range
      f[lane] = r.w0 * r.tok * weight;
      f[TB + lane] = r.w1 * r.tok * weight;
      f[2 * TB + lane] = r.w2 * r.tok * weight;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(b.accf(acc.slot));
    acc.next(kAccBufs);
  }
}

// ------------------------------------------------------------------ epilogue

// Four warps: thread r holds rows r and r + 128 of the tile (gate and up row of column
// r of the unit, or two output columns) for all tokens.
template <int TB>
struct Epilogue {
  const Block<TB>& b;
  const Fp8MoeArgs& a;
  const Routes& rt;
  int r;                                    // 0 .. 127
  uint32_t meets = 0;

  // All four warps (bounded: a warp may have given up).
  __device__ __forceinline__ bool meet() {
    mbar_arrive(b.meet());
    const bool ok = wait_soon(b.meet(), meets & 1u, b.ctl, b.status);
    ++meets;
    return __all_sync(kFullWarp, ok);
  }

  // h of the unit's column r for the expert's tokens, quantised over the unit's columns.
  __device__ __forceinline__ bool finish_h(int x, int unit, const float (&g)[TB],
                                           const float (&u)[TB]) {
    const int col = unit * 128 + r, warp = r >> 5, lane = r & 31;
    const uint32_t tokens = rt.tokens[x];
    const int nkb = (a.I + 127) / 128;
    float h[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      h[t] = 0.f;
      if (tokens >> t & 1u) {
        if (col < a.I) h[t] = g[t] / (1.f + __expf(-g[t])) * u[t];
        // magnitudes order as integers; a NaN counts as nothing
        const float m = fmaxf(fabsf(h[t]), 0.f);
        const uint32_t top = __reduce_max_sync(kFullWarp, __float_as_uint(m));
        if (lane == 0) b.red()[warp * TB + t] = __uint_as_float(top);
      }
    }
    if (!meet()) return false;
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      if (tokens >> t & 1u) {
        const float* m = b.red() + t;
        const BlockScale32 s(fmaxf(fmaxf(m[0], m[TB]), fmaxf(m[2 * TB], m[3 * TB])));
        if (col < a.I)
          a.hq[(static_cast<int64_t>(x) * TB + t) * a.ld_hq + col] =
              static_cast<uint8_t>(e4m3x4(s.quotient(h[t]), 0.f, 0.f, 0.f));
        if (r == 0) __stcg(a.hs + (static_cast<int64_t>(x) * nkb + unit) * TB + t, s.scale);
      }
    }
    return meet();                          // the maxima have been read
  }

  __device__ __forceinline__ void finish_out(int unit, const float (&v)[TB], const float (&w)[TB]) {
    const int c = unit * 256 + r;
    uint16_t* out = static_cast<uint16_t*>(a.out);
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      if (t < a.T) {
        if (c < a.N) out[t * a.ldo + c] = f32_to_out16(v[t], a.type);
        if (c + 128 < a.N) out[t * a.ldo + c + 128] = f32_to_out16(w[t], a.type);
      }
    }
  }

  // The block's tiles of an item are added up: the item is finished here, or by the last
  // block to come with its part.
  __device__ __forceinline__ bool finish(const Phase& p, int item, bool whole, float (&v)[TB],
                                         float (&w)[TB]) {
    const int x = p.down ? 0 : item / p.units;
    const int unit = p.down ? item : item % p.units;
    if (!whole) {
      const int c0 = p.owner(item * p.per_item), c1 = p.owner((item + 1) * p.per_item - 1);
      // A block's first item is its part 0, its last one (if another) its part 1: of an
      // item's blocks only the first can have begun with another.
      const int other = p.begin(c0) / p.per_item == item ? 0 : 1;
      auto part = [&](int block) {
        return a.part + (2 * block + (block == c0 ? other : 0)) * (2 * TB * 128) + r;
      };
      float* mine = part(static_cast<int>(blockIdx.x));
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        if (t < a.T) {
          __stcg(mine + t * 128, v[t]);
          __stcg(mine + (TB + t) * 128, w[t]);
        }
      }
      __threadfence();
      const uint32_t all = static_cast<uint32_t>(c1 - c0 + 1);
      uint32_t before = 0;
      if (p.down) {
        // output columns stand alone: the last of each warp's 64
        __syncwarp();
        if ((r & 31) == 0) before = atomicAdd(a.arrived + a.items1 + 4 * item + (r >> 5), 1u);
        before = __shfl_sync(kFullWarp, before, 0);
      } else {
        // a block of h is quantised together
        if (!meet()) return false;
        uint32_t* said = reinterpret_cast<uint32_t*>(b.red());
        if (r == 0) *said = atomicAdd(a.arrived + item, 1u);
        if (!meet()) return false;
        before = *said;
        if (!meet()) return false;          // it has been read
      }
      if (before + 1u != all) return true;
      __threadfence();
#pragma unroll
      for (int t = 0; t < TB; ++t) v[t] = w[t] = 0.f;
      // the parts in block order, 64 reads on their way (a read takes about 0.7 us)
      constexpr int kTogether = 32 / TB;
#pragma unroll 1
      for (int c = c0; c <= c1; c += kTogether) {
        float pv[kTogether][TB], pw[kTogether][TB];
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
          const float* q = part(min(c + i, c1));
#pragma unroll
          for (int t = 0; t < TB; ++t) {
            pv[i][t] = t < a.T ? __ldcg(q + t * 128) : 0.f;
            pw[i][t] = t < a.T ? __ldcg(q + (TB + t) * 128) : 0.f;
          }
        }
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
          if (c + i <= c1) {
#pragma unroll
            for (int t = 0; t < TB; ++t) { v[t] += pv[i][t]; w[t] += pw[i][t]; }
          }
        }
      }
    }
    if (p.down) {
      finish_out(unit, v, w);
      return true;
    }
    return finish_h(x, unit, v, w);
  }

  __device__ __forceinline__ bool run(const Phase& p, Ring& acc) {
    using S = Shape<TB>;
    const uint32_t lanes = b.tmem + (static_cast<uint32_t>(r >> 5) << 21);
    Cursor c;
    c.at(p, p.first);
    int item = p.first / p.per_item, inner = p.first - item * p.per_item;
    bool from_start = inner == 0;
    float v[TB], w[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) v[t] = w[t] = 0.f;
    for (int i = 0; i < p.count; ++i) {
      const bool ok = wait_soon(b.accf(acc.slot), acc.phase, b.ctl, b.status);
      if (!__all_sync(kFullWarp, ok)) return false;
      tc_fence_after();
      // which of the two scales of the second group: rows past a multiple of 128
      const int second =
          !p.down && (a.I + c.unit * 128 + r) / 128 != (a.I + c.unit * 128) / 128 ? 2 : 1;
      const uint32_t tokens = p.down ? rt.tokens[c.x] : ~0u;
      const float* f0 = b.fac(acc.slot);
      const float* f1 = f0 + second * TB;
#pragma unroll
      for (int t0 = 0; t0 < TB; t0 += 8) {
        uint32_t d[8], e[8];
        tmem_ld8(lanes + acc.slot * 2 * S::kCols + t0, d);
        tmem_ld8(lanes + acc.slot * 2 * S::kCols + S::kCols + t0, e);
        tmem_ld_wait();
        keep_after(d);
        keep_after(e);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          // a token that the expert does not have brings codes of no meaning
          if (tokens >> (t0 + t) & 1u) {
            v[t0 + t] = fmaf(__uint_as_float(d[t]), f0[t0 + t], v[t0 + t]);
            w[t0 + t] = fmaf(__uint_as_float(e[t]), f1[t0 + t], w[t0 + t]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(b.acce(acc.slot));
      acc.next(kAccBufs);
      c.next(p);
      if (++inner == p.per_item || i + 1 == p.count) {
        if (!finish(p, item, from_start && inner == p.per_item, v, w)) return false;
        if (inner == p.per_item) {
          inner = 0;
          ++item;
          from_start = true;
        }
#pragma unroll
        for (int t = 0; t < TB; ++t) v[t] = w[t] = 0.f;
      }
    }
    return true;
  }
};

// Logits of the block's experts: the threads share K, the weights' loads are issued
// together and a token's ahead of the one before it.
template <int DT, int RT, int TB>
__device__ __forceinline__ void router_logits(const Fp8MoeArgs& a, float (*part)[TB]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kChunks = 4, kPass = kThreads * 8 * kChunks;
  const int k0 = threadIdx.x * 8;
  for (int e = blockIdx.x; e < a.rule.E; e += gridDim.x) {
    for (int from = 0; from < a.K; from += kPass) {
      Pack<DT, 8> x[kChunks];
      float w[kChunks][8];
      auto load = [&](int t) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const int k = from + k0 + c * kThreads * 8;
          x[c].zero();
          if (k < a.K && t < a.T) x[c].load(a.x, t * a.ld + k);
        }
      };
      load(0);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int k = from + k0 + c * kThreads * 8;
        const int64_t at = static_cast<int64_t>(e) * a.K + k;
        if constexpr (RT == NVFP4_FP32) {
          Pack<NVFP4_FP32, 4> lo, hi;
          lo.zero();
          hi.zero();
          if (k < a.K) { lo.load(a.router, at); hi.load(a.router, at + 4); }
#pragma unroll
          for (int i = 0; i < 4; ++i) { w[c][i] = lo.get(i); w[c][4 + i] = hi.get(i); }
        } else {
          Pack<RT, 8> v;
          v.zero();
          if (k < a.K) v.load(a.router, at);
#pragma unroll
          for (int i = 0; i < 8; ++i) w[c][i] = v.get(i);
        }
      }
#pragma unroll 1
      for (int t = 0; t < a.T; ++t) {
        float sum[kChunks];
        Pack<DT, 8> now[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) now[c] = x[c];
        load(t + 1);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          sum[c] = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[c] = fmaf(now[c].get(i), w[c][i], sum[c]);
        }
        const float v = warp_sum((sum[0] + sum[1]) + (sum[2] + sum[3]));
        if (lane == 0) part[warp][t] = from == 0 ? v : part[warp][t] + v;
      }
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
__device__ __forceinline__ void gate_token(const Fp8MoeArgs& a, Routes& rt, int t) {
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

// The routes by expert, the same in every block: an expert's tokens are the bits of a
// word, a route's place among the expert's the bits below its own.
__device__ __forceinline__ void list_experts(const Fp8MoeArgs& a, Routes& rt, uint32_t* bits,
                                             int2* scan) {
  const int topk = a.rule.topk, R = a.T * topk;
  const int r = threadIdx.x, warp = r >> 5, lane = r & 31;
  for (int i = r; i < a.rule.E; i += kThreads) bits[i] = 0;
  if (!a.router && r < a.T) {
    // an expert that a token names twice: once, with both weights
    const int i = r * topk;
#pragma unroll 1
    for (int k = 1; k < topk; ++k)
#pragma unroll 1
      for (int j = 0; j < k; ++j)
        if (rt.expert[i + k] >= 0 && rt.expert[i + k] == rt.expert[i + j]) {
          rt.weight[i + j] += rt.weight[i + k];
          rt.expert[i + k] = -1;
        }
  }
  __syncthreads();
  const int e = r < R ? rt.expert[r] : -1;
  const int t = r / topk;
  if (e >= 0) atomicOr(bits + e, 1u << t);
  __syncthreads();
  const uint32_t tokens = e >= 0 ? bits[e] : 0u;
  const uint32_t below = e >= 0 ? tokens & ((1u << t) - 1u) : 0u;
  const bool lead = e >= 0 && below == 0;
  // exclusive sums over the leading routes: experts (x) and entries (y)
  int2 v = make_int2(lead ? 1 : 0, lead ? __popc(tokens) : 0);
  const int2 own = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFullWarp, v.x, o), y = __shfl_up_sync(kFullWarp, v.y, o);
    if (lane >= o) { v.x += x; v.y += y; }
  }
  if (lane == 31) scan[warp] = v;
  __syncthreads();
  int2 base = make_int2(v.x - own.x, v.y - own.y);
#pragma unroll 1
  for (int w = 0; w < warp; ++w) { base.x += scan[w].x; base.y += scan[w].y; }
  if (lead) {
    rt.live[base.x] = static_cast<int16_t>(e);
    rt.start[base.x] = static_cast<int16_t>(base.y);
    rt.tokens[base.x] = tokens;
    bits[e] = base.y;                       // from here on: the expert's first entry
  }
  if (r == kThreads - 1) rt.n_live = base.x + own.x;
  __syncthreads();
  if (e >= 0) rt.route[bits[e] + __popc(below)] = static_cast<int16_t>(r);
  __syncthreads();
}

// Rows of x as codes and scales in the workspace, spread over the grid's warps from the
// last block on (the first ones have the router's experts).
template <int DT>
__device__ __forceinline__ void quantise_tokens(const Fp8MoeArgs& a, int columns) {
  const int lane = threadIdx.x & 31;
  const int chunks = (a.K + 511) / 512;
  for (int i = (threadIdx.x >> 5) * gridDim.x + gridDim.x - 1 - blockIdx.x; i < a.T * chunks;
       i += kWarps * gridDim.x) {
    const int t = i / chunks, k = (i - t * chunks) * 512 + lane * 16;
    float v[16];
    if (k < a.K) {
      load_row16<DT, false>(a.x, t * a.ld, a.K, k, v);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.f;
    }
    const BlockScale s(block_amax(v));
    if (k >= a.K) continue;
    uint4 q;
    uint32_t* qw = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      qw[j] = e4m3x4(s.quotient(v[4 * j]), s.quotient(v[4 * j + 1]), s.quotient(v[4 * j + 2]),
                     s.quotient(v[4 * j + 3]));
    *reinterpret_cast<uint4*>(a.xq + t * a.ld_xq + k) = q;
    if ((lane & 7) == 0) __stcg(a.xs + (k / kFp8Block) * columns + t, s.scale);
  }
}

// What the first barrier waits for.
template <int DT, int TB>
__device__ __forceinline__ void before_gate(const Fp8MoeArgs& a, float (*part)[TB]) {
  quantise_tokens<DT>(a, TB);
  if (!a.router) return;
  if (a.router_type == NVFP4_FP32) router_logits<DT, NVFP4_FP32, TB>(a, part);
  else router_logits<DT, DT, TB>(a, part);
}

template <int TB>
__global__ void __launch_bounds__(kThreads, 1)
fp8_moe_kernel(const __grid_constant__ CUtensorMap t1, const __grid_constant__ CUtensorMap t2,
               const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap th,
               const __grid_constant__ Fp8MoeArgs a) {
  using S = Shape<TB>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Routes rt;
  __shared__ float part[kWarps][TB];
  __shared__ int2 scan[kWarps];
  __shared__ uint32_t bits[kGateMaxExperts];
  Block<TB> b;
  b.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~static_cast<uintptr_t>(1023));
  b.base = smem_u32(b.smem);
  b.ctl = reinterpret_cast<CtaCtl*>(b.smem + S::kCtlOffset);
  b.status = a.status;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(b.smem + S::kCtlOffset + 16);
  const int warp = threadIdx.x >> 5;
  cg::grid_group grid = cg::this_grid();

  if (threadIdx.x == 0) {
    prefetch_map(&t1);
    prefetch_map(&t2);
    prefetch_map(&tx);
    prefetch_map(&th);
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(b.full(s), 1);
      mbar_init(b.empty(s), 1);
    }
    for (int i = 0; i < kAccBufs; ++i) {
      mbar_init(b.accf(i), 2);                  // the sums, and the factors
      mbar_init(b.acce(i), 4);
    }
    mbar_init(b.drain(), 1);
    mbar_init(b.meet(), 128);
    b.ctl->abort = 0;
    b.ctl->timeout_ns = a.timeout_ns;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), S::kTmemCols);
    tmem_relinquish();
  }
  const int units1 = (a.I + 127) / 128, units2 = (a.N + 255) / 256;
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < a.items1 + 4 * units2;
       i += gridDim.x * kThreads)
    __stcg(a.arrived + i, 0u);
  if (a.type == NVFP4_BF16) before_gate<NVFP4_BF16, TB>(a, part);
  else before_gate<NVFP4_FP16, TB>(a, part);
  fence_proxy_async_global();                   // the codes are read by TMA
  tc_fence_before();
  grid.sync();
  tc_fence_after();
  b.tmem = *tmem_slot;

  if (a.router) {
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
  list_experts(a, rt, bits, scan);

  Phase p1, p2;
  p1.set(0, (a.K + 127) / 128, units1, rt.n_live);
  p2.set(1, (a.I + 127) / 128, units2, rt.n_live);
  const int early = min(S::kStages, p2.count);  // down tiles whose weights go ahead
  Ring ring, acc;
  const uint32_t idesc = idesc_e4m3(128, S::kCols);
  const bool lead = warp < 2 && elect_one();
  Cursor c;
  uint32_t issued = 0;
  bool alive = true;

  auto multiply = [&](const Phase& p) {
    for (int i = 0; i < p.count && alive; ++i) {
      if (!wait_both(b.acce(acc.slot), acc.phase ^ 1u, b.full(ring.slot), ring.phase, b.ctl,
                     b.status)) {
        alive = false;
        break;
      }
      tc_fence_after();
      const uint32_t s = b.stage(ring.slot), d = b.tmem + acc.slot * 2 * S::kCols;
      const uint64_t tok = sdesc_sw128(s + S::kTokOffset);
      tc_mma_e4m3_k128(d, sdesc_sw128(s), tok, idesc);
      tc_mma_e4m3_k128(d + S::kCols, sdesc_sw128(s + kGroupBytes), tok, idesc);
      tc_commit(b.accf(acc.slot));
      tc_commit(b.empty(ring.slot));
      ring.next(S::kStages);
      acc.next(kAccBufs);
    }
  };
  Epilogue<TB> epi{b, a, rt, static_cast<int>(threadIdx.x) & 127};

  // ------------------------------------------------------------------ gate_up
  if (warp == 0) {
    if (lead) {
      fence_proxy_async_global();
      const Producer<TB> first{b, rt, &t1, &tx, l2_policy_evict_first(), l2_policy_evict_last()};
      c.at(p1, p1.first);
      for (int i = 0; i < p1.count; ++i) {
        if (!wait_soon(b.empty(ring.slot), ring.phase ^ 1u, b.ctl, b.status)) {
          alive = false;
          break;
        }
        first.weights(p1, c, ring.slot);
        first.tokens(p1, c, ring.slot);
        ++issued;
        ring.next(S::kStages);
        c.next(p1);
      }
      // down weights as the stages come free: they need no h
      const Producer<TB> then{b, rt, &t2, &th, first.wpol, first.tpol};
      Ring r = ring;
      c.at(p2, p2.first);
      for (int i = 0; i < early && alive; ++i) {
        if (!wait_soon(b.empty(r.slot), r.phase ^ 1u, b.ctl, b.status)) {
          alive = false;
          break;
        }
        then.weights(p2, c, r.slot);
        ++issued;
        r.next(S::kStages);
        c.next(p2);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lead) multiply(p1);
    __syncwarp();
  } else if (warp == 2) {
    factors<TB>(b, a, rt, p1, acc);
  } else if (warp >= 4) {
    alive = epi.run(p1, acc);
    fence_proxy_async_global();                 // so are the codes of h
  }
  grid.sync();

  // --------------------------------------------------------------------- down
  if (warp == 0) {
    if (lead) {
      fence_proxy_async_global();
      const Producer<TB> then{b, rt, &t2, &th, l2_policy_evict_first(), l2_policy_evict_last()};
      c.at(p2, p2.first);
      for (int i = 0; i < p2.count; ++i) {
        if (i >= early) {
          if (!alive || !wait_soon(b.empty(ring.slot), ring.phase ^ 1u, b.ctl, b.status)) break;
          then.weights(p2, c, ring.slot);
          ++issued;
        } else if (!alive) {
          break;
        }
        then.tokens(p2, c, ring.slot);
        ring.next(S::kStages);
        c.next(p2);
      }
      // what is on its way lands before the shared memory goes away
      const uint32_t late = issued > static_cast<uint32_t>(S::kStages) ? issued - S::kStages : 0u;
      for (uint32_t i = late; i < issued; ++i)
        wait_drain(b.full(static_cast<int>(i % S::kStages)), (i / S::kStages) & 1u,
                   b.ctl->timeout_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lead) {
      multiply(p2);
      tc_commit(b.drain());
      wait_drain(b.drain(), 0, b.ctl->timeout_ns);
    }
    __syncwarp();
  } else if (warp == 2) {
    factors<TB>(b, a, rt, p2, acc);
  } else if (warp >= 4) {
    if (alive) epi.run(p2, acc);
  }
  if (rt.n_live == 0)                           // no route at all
    for (int64_t i = blockIdx.x * kThreads + threadIdx.x; i < static_cast<int64_t>(a.T) * a.N;
         i += static_cast<int64_t>(gridDim.x) * kThreads)
      static_cast<uint16_t*>(a.out)[i / a.N * a.ldo + i % a.N] = 0;
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(b.tmem, S::kTmemCols);
  }
}

template <int TB>
cudaError_t go(const CUtensorMap& t1, const CUtensorMap& t2, const CUtensorMap& tx,
               const CUtensorMap& th, const Fp8MoeArgs& a, int sms, cudaStream_t s) {
  void* args[] = {const_cast<CUtensorMap*>(&t1), const_cast<CUtensorMap*>(&t2),
                  const_cast<CUtensorMap*>(&tx), const_cast<CUtensorMap*>(&th),
                  const_cast<Fp8MoeArgs*>(&a)};
  return cudaLaunchCooperativeKernel(fp8_moe_kernel<TB>,
                                     dim3(sms < kMoeMaxGrid ? sms : kMoeMaxGrid), dim3(kThreads),
                                     args, Shape<TB>::kSmemBytes, s);
}

template <int TB>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(fp8_moe_kernel<TB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Shape<TB>::kSmemBytes);
}

}  // namespace

cudaError_t init_fp8_moe_attributes() {
  cudaError_t e = set_smem<8>();
  if (e == cudaSuccess) e = set_smem<16>();
  if (e == cudaSuccess) e = set_smem<32>();
  return e;
}

int fp8_moe_box_rows(int columns) { return columns < 16 ? 16 : columns; }

bool fp8_moe_layout(int64_t T, int32_t topk, int32_t E, int64_t K, int64_t I, int64_t N,
                    MoeLayout* m) {
  if (T <= 0 || topk <= 0 || E <= 0 || topk > E || K <= 0 || I <= 0 || N <= 0 || K % 16 != 0 ||
      I % 16 != 0 || T > kMoeMaxTokens || T * topk > kMoeMaxRoutes || E > kGateMaxExperts ||
      topk > kGateMaxTopk || K > (1 << 20) || I > (1 << 20) || N > (1 << 20))
    return false;
  const int64_t R = T * topk;
  const int64_t live = R < E ? R : E, kx = (K + 127) / 128, kh = (I + 127) / 128;
  const int64_t units2 = (N + 255) / 256;
  if (live * kh * kx > 0x3FFFFFFF || live * kh * units2 > 0x3FFFFFFF) return false;   // tiles
  size_t end = 0;
  auto take = [&](int64_t bytes) {
    const size_t at = end;
    end += static_cast<size_t>((bytes + 255) / 256 * 256);
    return at;
  };
  m->columns = T > 16 ? 32 : T > 8 ? 16 : 8;
  m->experts = static_cast<int>(live);
  m->ld_xq = kx * 128;
  m->ld_hq = kh * 128;
  take(T * E * 4);
  m->xq = take(m->columns * m->ld_xq);
  m->xs = take(kx * m->columns * 4);
  m->hq = take(live * m->columns * m->ld_hq);
  m->hs = take(live * kh * m->columns * 4);
  m->part = take(static_cast<int64_t>(2) * kMoeMaxGrid * 2 * m->columns * 128 * 4);
  m->arrived = take((live * kh + 4 * units2) * 4);
  m->bytes = end;
  return true;
}

cudaError_t launch_fp8_moe(const CUtensorMap& t1, const CUtensorMap& t2, const CUtensorMap& tx,
                           const CUtensorMap& th, const Fp8MoeArgs& a, int columns, int sms,
                           cudaStream_t s) {
  switch (columns) {
    case 8: return go<8>(t1, t2, tx, th, a, sms, s);
    case 16: return go<16>(t1, t2, tx, th, a, sms, s);
    default: return go<32>(t1, t2, tx, th, a, sms, s);
  }
}

}  // namespace nvfp4
