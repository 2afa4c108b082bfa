// A whole MoE layer for a few tokens (up to 8) over FP8 experts:
//
//   l = x . router^T;  experts e_tk and weights w_tk by the top-k gate (gate.cuh)
//   h_tk = SiLU(xq . gate_e^T) * (xq . up_e^T),   out_t = sum_k w_tk hq_tk . down_e^T
//
// with xq and hq the rows' E4M3 codes with 1 x 128 scales (fp8_quant.cuh; h from FP32)
// and FP32 sums in a fixed order: results repeat bit for bit.
//
// Bound: the chosen experts' bytes (HBM).  The design serves that stream:
//
// * Two launches.  The first, small one writes the logits (router rows spread over the
//   blocks) and the codes of x; the second is launched to overlap it and waits for it with
//   its set-up done.  Every block of the second makes the choice for itself.
// * Weights are the MMA's 128 rows (tcgen05, M 128), the tokens half of its 16 columns: all
//   tokens, so that nothing is gathered; an expert's columns of other tokens are dropped.
//   A tile is 256 weight rows x 128 K (32 KB, two TMA boxes): the gate and up rows of 128
//   columns of h, so that one thread holds both factors of its h, or 256 down rows.
//   Rows past a matrix read as zeros.
// * The tiles of a phase stand in one line (gate_up: expert, 128 columns, K block; down:
//   256 columns, expert, K block) that is cut into equal runs, as many as blocks, wherever
//   that falls: a token's eight experts have some thousands of tiles, and every SM streams
//   the same bytes.  An item (128 columns of one expert's h; 256 output columns over all
//   experts) whose tiles lie in several runs is joined by the last run to finish, which
//   adds the parts in the order of the runs.  (Two to eight shorter runs a block, for SMs that
//   are not equally fast: the joins cost more, 8 tokens 308 -> 311 to 333 us.)
// * Blocks take runs by a counter, all of gate_up's before the first of down's, and a down
//   run waits (bounded) until all gate_up runs are done.  Those are then in the hands of
//   blocks that run, so that no block has to wait for one that has not started: a plain
//   launch, whatever else is on the GPU.
// * Six stages are on their way (192 KB an SM).  When a block has asked for all its gate_up
//   tiles, its producer takes its down run and goes on with the weights of the first down
//   tiles, before it waits for the codes of h: HBM does not idle there.
// * Both scales differ by K block, so every K block has accumulators of its own in tensor
//   memory, which four warps read and add as FP32 times the factor (weight scale * token
//   scale, for down also * routing weight) that a warp of its own lays out.
//
// Measured in a graph, 128 experts, 8 chosen: 6144 x 2048 one token 61 us (302 MB of weights,
// 0.73 of the copy rate; about 7 us pass before the first weights are asked for, and 6 behind
// the last ones), 2 tokens 108, 4 tokens 178, 8 tokens 305 us (1.9 GB, 0.93); 2048 x 768 26, 33,
// 47 and 61 us.  A first form with mma.sync, eight warps with rings of their own, spent 280
// instructions on 2 KB of weights, converting codes: one token 96 us.  One cooperative launch
// with the router in it, between grid barriers, instead of the two: 68 us.
#include "fp8_common.cuh"
#include "fp8_moe.h"
#include "fp8_quant.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroupBytes = 128 * 128;      // 128 weight rows of a K block
constexpr int kAccBufs = 8;                 // of 2 x 16 columns

constexpr int TB = kMoeMaxTokens;           // token columns that are read
constexpr int kCols = 16;                   // of the MMA: its fewest
constexpr int kStages = 6;
constexpr int kTokOffset = 2 * kGroupBytes;
constexpr int kStageBytes = kTokOffset + kCols * 128;
constexpr int kFacOffset = kStages * kStageBytes;           // [bufs][3][TB] floats
constexpr int kRedOffset = kFacOffset + kAccBufs * 3 * TB * 4;   // [4][TB] maxima
constexpr int kBarOffset = kRedOffset + 4 * TB * 4;
constexpr int kCtlOffset = kBarOffset + 8 * (2 * kStages + 2 * kAccBufs + 7);
constexpr int kSmemBytes = kCtlOffset + 32 + 1024;
constexpr uint32_t kTmemCols = kAccBufs * 2 * kCols;

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

__device__ __forceinline__ void ld_shared8(uint32_t addr, float (&f)[8]) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]) : "r"(addr) : "memory");
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7]) : "r"(addr + 16) : "memory");
}

// Uses of r stay behind the wait for its load (volatile statements keep their order).
__device__ __forceinline__ void keep_after(uint32_t (&r)[8]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                    "+r"(r[6]), "+r"(r[7]));
}

// One phase's line of tiles, cut into runs.
struct Phase {
  int down;
  int nkb;                                  // K blocks of an item's expert
  int units;                                // gate_up: ceil(I / 128); down: ceil(N / 256)
  int experts;
  int per_item;                             // tiles of an item
  int grain, grains;                        // runs begin at multiples of `grain` tiles
  int parts;                                // runs

  // (the host refuses sizes whose tiles times runs pass 32 bits)
  __device__ __forceinline__ int begin(int run) const {
    return grain * static_cast<int>(static_cast<uint32_t>(grains) * run / static_cast<uint32_t>(parts));
  }
  // The run that holds a tile.
  __device__ __forceinline__ int owner(int tile) const {
    return static_cast<int>(((static_cast<uint32_t>(tile) / grain + 1) * parts - 1) /
                            static_cast<uint32_t>(grains));
  }
  // Runs of whole items need no join, which takes about 4 us behind the last tile; runs of
  // single tiles are all equally long.  A tile takes 0.76 us while all SMs draw on HBM and
  // at least 0.53 us (62 GB/s is all that one SM draws); a join 5 tiles' time and
  // a third of one for each part, since the last run reads them all: an item of n tiles is cut
  // into about sqrt(1.5 n) runs, eight at least (8 tokens, 39 experts of 512 x 2048, whose down
  // items have 624 tiles: 75 -> 48 us; eight are best for small items).  As many runs of each
  // item where that leaves no more than a fifth of the blocks idle: none then has parts of
  // two items (one token, 4 experts of 4096 x 1024: 29 -> 26 us).
  __device__ __forceinline__ void set(int is_down, int k_blocks, int n_units, int n_experts) {
    const int blocks = static_cast<int>(gridDim.x);
    down = is_down;
    nkb = k_blocks;
    units = n_units;
    experts = n_experts;
    per_item = max(down ? nkb * experts : nkb, 1);
    const int items = down ? units * min(experts, 1) : units * experts;
    const int rest = items % blocks;
    // (in floating point: the products can pass 32 bits)
    const float rounds = static_cast<float>(items / blocks) +
                         (rest ? fmaxf(0.7f, static_cast<float>(rest) / blocks) : 0.f);
    const bool whole = rounds * per_item <= static_cast<float>(items) * per_item / blocks + 5.f;
    grain = whole ? per_item : 1;
    grains = whole ? items : items * per_item;
    const int share = max(8, static_cast<int>(sqrtf(1.5f * static_cast<float>(per_item))));
    parts = min(blocks, min(grains, share * items));
    if (!whole && parts == blocks) {
      const int even = blocks / items * items;
      if (5 * even >= 4 * blocks) parts = even;
    }
  }
};

// A run that the block has taken.
struct Run {
  int phase;                                // 2: no more
  int number, first, count;
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
struct Block {
  uint32_t base;
  uint8_t* smem;
  CtaCtl* ctl;
  int* status;
  uint32_t tmem;
  __device__ __forceinline__ uint32_t stage(int s) const { return base + s * kStageBytes; }
  __device__ __forceinline__ uint32_t bar(int i) const { return base + kBarOffset + 8u * i; }
  __device__ __forceinline__ uint32_t full(int s) const { return bar(s); }
  __device__ __forceinline__ uint32_t empty(int s) const { return bar(kStages + s); }
  __device__ __forceinline__ uint32_t accf(int b) const { return bar(2 * kStages + b); }
  __device__ __forceinline__ uint32_t acce(int b) const {
    return bar(2 * kStages + kAccBufs + b);
  }
  __device__ __forceinline__ uint32_t drain() const { return bar(2 * kStages + 2 * kAccBufs); }
  __device__ __forceinline__ uint32_t meet() const {
    return bar(2 * kStages + 2 * kAccBufs + 1);
  }
  __device__ __forceinline__ uint32_t run_given(int i) const {
    return bar(2 * kStages + 2 * kAccBufs + 2 + i);
  }
  __device__ __forceinline__ uint32_t run_taken(int i) const {
    return bar(2 * kStages + 2 * kAccBufs + 4 + i);
  }
  __device__ __forceinline__ uint32_t chosen() const {
    return bar(2 * kStages + 2 * kAccBufs + 6);
  }
  __device__ __forceinline__ float* fac(int b) const {
    return reinterpret_cast<float*>(smem + kFacOffset) + b * 3 * TB;
  }
  __device__ __forceinline__ uint32_t fac_at(int i) const {
    return base + kFacOffset + i * 3 * TB * 4;
  }
  __device__ __forceinline__ float* red() const {
    return reinterpret_cast<float*>(smem + kRedOffset);
  }
};

// What the roles of a block wait on for their next run: the producer takes it, the MMA's
// lane, the factors' warp and the four warps of the epilogue each read it once.
constexpr int kRunReaders = 6;

struct Runs {
  const Block& b;
  Run* slots;                               // [2]
  uint32_t n = 0;
  __device__ __forceinline__ bool give(const Run& r) {
    if (!wait_soon(b.run_taken(n & 1u), (n >> 1 & 1u) ^ 1u, b.ctl, b.status)) return false;
    slots[n & 1u] = r;
    mbar_arrive(b.run_given(n & 1u));
    ++n;
    return true;
  }
  // `whole`: by all lanes of a warp.
  __device__ __forceinline__ bool take(Run* r, bool whole) {
    bool ok = wait_soon(b.run_given(n & 1u), n >> 1 & 1u, b.ctl, b.status);
    if (whole) ok = __all_sync(kFullWarp, ok);
    if (!ok) return false;
    *r = slots[n & 1u];
    if (whole) __syncwarp();
    if (!whole || (threadIdx.x & 31) == 0) mbar_arrive(b.run_taken(n & 1u));
    ++n;
    return true;
  }
};

// Waits (acquire) until *p >= target; bounded like the other waits.
__device__ __forceinline__ bool wait_runs(const uint32_t* p, uint32_t target, CtaCtl* ctl,
                                          int* status) {
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 0; i < 0x7FFFFFFFu; ++i) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    if (v >= target) return true;
    if (*reinterpret_cast<volatile uint32_t*>(&ctl->abort)) return false;
    if (globaltimer() - t0 > ctl->timeout_ns) break;
    __nanosleep(32);
  }
  *reinterpret_cast<volatile uint32_t*>(&ctl->abort) = 1u;
  raise_status(status, NVFP4_ERR_TIMEOUT);
  return false;
}

// Counts a role's passes over a ring of n slots.
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) { slot = 0; phase ^= 1u; }
  }
};

// ------------------------------------------------------------------ producer

struct Producer {
  const Block& b;
  const Routes& rt;
  const CUtensorMap* w;
  const CUtensorMap* tok;
  uint64_t wpol, tpol;

  __device__ __forceinline__ void weights(const Phase& p, const Cursor& c, int s) const {
    const int e = rt.live[c.x];
    mbar_arrive_expect_tx(b.full(s), kStageBytes);
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
    tma_load_2d(b.stage(s) + kTokOffset, tok, b.full(s), c.kb * 128,
                p.down ? c.x * TB : 0, tpol);
  }
};

// ------------------------------------------------------------------- factors

// One warp: for each tile the products of the weight scales (gate or first 128 rows; up
// or second 128 rows, whose scale can change within the 128 rows where I is no multiple
// of 128) and of each token's scale (times its routing weight in the down phase).
__device__ __forceinline__ void factors(const Block& b, const Fp8MoeArgs& a, const Routes& rt,
                                        const Phase& p, const Run& run, Ring& acc) {
  const int lane = threadIdx.x & 31;
  Cursor c;
  c.at(p, run.first);
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
  Raw next = load(c);
#pragma unroll 1
  for (int i = 0; i < run.count; ++i) {
    const Raw r = next;
    if (p.down && c.x != x) {
      x = c.x;
      const uint32_t tokens = rt.tokens[x];
      const int j = rt.start[x] + __popc(tokens & ((1u << lane) - 1u));
      weight = tokens >> lane & 1u ? rt.weight[rt.route[j]] : 0.f;
    }
    c.next(p);
    if (i + 1 < run.count) next = load(c);
    if (!__all_sync(kFullWarp, wait_soon(b.acce(acc.slot), acc.phase ^ 1u, b.ctl, b.status)))
      return;
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
struct Epilogue {
  const Block& b;
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

  // h of the unit's column r for one of the expert's tokens.
  __device__ __forceinline__ float h_of(const float (&g)[TB], const float (&u)[TB], int token,
                                        bool in) const {
    float gate = 0.f, up = 0.f;
#pragma unroll
    for (int t = 0; t < TB; ++t)
      if (t == token) { gate = g[t]; up = u[t]; }
    return in ? gate / (1.f + __expf(-gate)) * up : 0.f;
  }
  // The unit's columns of h for the expert's tokens, quantised together.  (A loop over the
  // tokens: unrolled, its instructions took longer to fetch than to run.)
  __device__ __forceinline__ bool finish_h(int x, int unit, uint32_t tokens, const float (&g)[TB],
                                           const float (&u)[TB]) {
    const int col = unit * 128 + r, warp = r >> 5;
    const bool in = col < a.I;
#pragma unroll 1
    for (uint32_t m = tokens; m; m &= m - 1) {
      const int t = __ffs(m) - 1;
      // magnitudes order as integers; a NaN counts as nothing
      const float top = fmaxf(fabsf(h_of(g, u, t, in)), 0.f);
      const uint32_t most = __reduce_max_sync(kFullWarp, __float_as_uint(top));
      if ((r & 31) == 0) b.red()[warp * TB + t] = __uint_as_float(most);
    }
    if (!meet()) return false;
#pragma unroll 1
    for (uint32_t m = tokens; m; m &= m - 1) {
      const int t = __ffs(m) - 1;
      const float* top = b.red() + t;
      const BlockScale32 s(fmaxf(fmaxf(top[0], top[TB]), fmaxf(top[2 * TB], top[3 * TB])));
      if (in)
        a.hq[(static_cast<int64_t>(x) * TB + t) * a.ld_hq + col] =
            static_cast<uint8_t>(e4m3x4(s.quotient(h_of(g, u, t, in)), 0.f, 0.f, 0.f));
      if (r == 0)
        __stcg(a.hs + (static_cast<int64_t>(x) * ((a.I + 127) / 128) + unit) * TB + t, s.scale);
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

  // A run's tiles of an item are added up: the item is finished here, or by the last run to
  // come with its part.
  __device__ __forceinline__ bool finish(const Phase& p, const Run& run, int item, int x, int unit,
                                         bool whole, float (&v)[TB], float (&w)[TB]) {
    if (!whole) {
      const int c0 = p.owner(item * p.per_item), c1 = p.owner((item + 1) * p.per_item - 1);
      // A run's first item is its part 0, its last one (if another) its part 1: of an
      // item's runs only the first can have begun with another.
      const int other = p.begin(c0) / p.per_item == item ? 0 : 1;
      auto part = [&](int number) {
        return a.part + (2 * number + (number == c0 ? other : 0)) * (2 * TB * 128) + r;
      };
      float* mine = part(run.number);
      const uint32_t tokens = p.down ? (1u << a.T) - 1u : rt.tokens[x];
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        if (tokens >> t & 1u) {
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
        if ((r & 31) == 0) before = atomicAdd(a.counters + 4 + a.items1 + 4 * item + (r >> 5), 1u);
        before = __shfl_sync(kFullWarp, before, 0);
      } else {
        // a block of h is quantised together
        if (!meet()) return false;
        uint32_t* said = reinterpret_cast<uint32_t*>(b.red());
        if (r == 0) *said = atomicAdd(a.counters + 4 + item, 1u);
        if (!meet()) return false;
        before = *said;
        if (!meet()) return false;          // it has been read
      }
      if (before + 1u != all) return true;
      __threadfence();
#pragma unroll
      for (int t = 0; t < TB; ++t) v[t] = w[t] = 0.f;
      // the parts in the order of the runs, 64 reads on their way (a read takes about 0.7 us)
      constexpr int kTogether = 4;
#pragma unroll 1
      for (int c = c0; c <= c1; c += kTogether) {
        float pv[kTogether][TB], pw[kTogether][TB];
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
          const float* q = part(min(c + i, c1));
#pragma unroll
          for (int t = 0; t < TB; ++t) {
            pv[i][t] = tokens >> t & 1u ? __ldcg(q + t * 128) : 0.f;
            pw[i][t] = tokens >> t & 1u ? __ldcg(q + (TB + t) * 128) : 0.f;
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
    return finish_h(x, unit, x < rt.n_live ? rt.tokens[x] : 1u, v, w);
  }

  __device__ __forceinline__ bool add(const Phase& p, const Run& run, Ring& acc, bool warm) {
    const uint32_t lanes = b.tmem + (static_cast<uint32_t>(r >> 5) << 21);
    Cursor c;
    c.at(p, run.first);
    int item = run.first / p.per_item, inner = run.first - item * p.per_item;
    bool from_start = inner == 0;
    float v[TB], w[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) v[t] = w[t] = 0.f;
    // Step -1 (warm), while the first weights are on their way: an item of zeros for an
    // expert that is none, so that what ends an item is in the instruction cache when the
    // first one does (5 us behind the last tile otherwise).
#pragma unroll 1
    for (int i = warm ? -1 : 0; i < run.count; ++i) {
      if (i >= 0) {
        const bool ok = wait_soon(b.accf(acc.slot), acc.phase, b.ctl, b.status);
        if (!__all_sync(kFullWarp, ok)) return false;
        tc_fence_after();
        // which of the two scales of the second group: rows past a multiple of 128
        const int second =
            !p.down && (a.I + c.unit * 128 + r) / 128 != (a.I + c.unit * 128) / 128 ? 2 : 1;
        const uint32_t f0 = b.fac_at(acc.slot), f1 = f0 + 4 * second * TB;
        const uint32_t tokens = rt.tokens[c.x];
        uint32_t d[TB], e[TB];
        tmem_ld8(lanes + acc.slot * 2 * kCols, d);
        tmem_ld8(lanes + acc.slot * 2 * kCols + kCols, e);
        float fd[TB], fe[TB];
        ld_shared8(f0, fd);
        ld_shared8(f1, fe);
        tmem_ld_wait();
        keep_after(d);
        keep_after(e);
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          // the columns of other tokens: in the down phase products with codes of no meaning
          if (tokens >> t & 1u) {
            v[t] = fmaf(__uint_as_float(d[t]), fd[t], v[t]);
            w[t] = fmaf(__uint_as_float(e[t]), fe[t], w[t]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(b.acce(acc.slot));
        acc.next(kAccBufs);
        c.next(p);
        ++inner;
      }
      if (i < 0 || inner == p.per_item || i + 1 == run.count) {
        const int x = i < 0 ? a.experts : p.down ? 0 : item / p.units;
        const int unit = i < 0 ? 0 : p.down ? item : item - x * p.units;
        if (!finish(p, run, item, x, unit, i < 0 || (from_start && inner == p.per_item), v, w))
          return false;
        if (i >= 0 && inner == p.per_item) {
          inner = 0;
          ++item;
          from_start = true;
        }
#pragma unroll
        for (int t = 0; t < TB; ++t) v[t] = w[t] = 0.f;
      }
    }
    if (!p.down) {
      // the run is done: its codes of h are read by TMA and by other blocks
      fence_proxy_async_global();
      __threadfence();
      if (!meet()) return false;
      if (r == 0)
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" :: "l"(a.counters + 2) : "memory");
    }
    return true;
  }
};

// Logits, a router's row and up to four tokens at a time: the threads share K, three
// 8-element chunks each, with the loads of the row and of the tokens on their way together.
template <int DT, int RT>
__device__ __forceinline__ void router_logits(const Fp8MoeArgs& a, float (*part)[4]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kChunks = 3, kTogether = 4, N = elems_per_16b<RT>();
  const int sets = (a.T + kTogether - 1) / kTogether;
  for (int i = blockIdx.x; i < a.rule.E * sets; i += gridDim.x) {
    const int e = i % a.rule.E, t0 = i / a.rule.E * kTogether;
    float sum[kTogether] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int from = threadIdx.x * 8; from < a.K; from += kThreads * 8 * kChunks) {
      Pack<RT, N> w[kChunks][8 / N];
      Pack<DT, 8> x[kTogether][kChunks];
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int k = from + c * kThreads * 8;
#pragma unroll
        for (int j = 0; j < 8 / N; ++j) {
          w[c][j].zero();
          if (k < a.K) w[c][j].load(a.router, static_cast<int64_t>(e) * a.K + k + j * N);
        }
#pragma unroll
        for (int t = 0; t < kTogether; ++t) {
          x[t][c].zero();
          if (t0 + t < a.T && k < a.K) x[t][c].load(a.x, (t0 + t) * a.ld + k);
        }
      }
#pragma unroll
      for (int t = 0; t < kTogether; ++t) {
        if (t0 + t >= a.T) break;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          float dot = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) dot = fmaf(x[t][c].get(j), w[c][j / N].get(j % N), dot);
          sum[t] += dot;
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kTogether; ++t) {
      if (t0 + t >= a.T) break;
      sum[t] = warp_sum(sum[t]);
      if (lane == 0) part[warp][t] = sum[t];
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < kTogether && t0 + t < a.T) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += part[w][t];
      __stcg(a.logits + static_cast<int64_t>(t0 + t) * a.rule.E + e, v);
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
    if (a.T == 1) rt.live[r] = static_cast<int16_t>(id);       // distinct ones
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
__device__ __forceinline__ void quantise_tokens(const Fp8MoeArgs& a) {
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
    if ((lane & 7) == 0) __stcg(a.xs + (k / kFp8Block) * TB + t, s.scale);
  }
}

// The first launch.
template <int DT>
__global__ void __maxnreg__(96) fp8_moe_router_kernel(const Fp8MoeArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float part[kWarps][4];
  const int counters = 4 + a.items1 + 4 * ((a.N + 255) / 256);
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < counters; i += gridDim.x * kThreads)
    a.counters[i] = 0u;
  quantise_tokens<DT>(a);
  if (!a.router) return;
  if (a.router_type == NVFP4_FP32) router_logits<DT, NVFP4_FP32>(a, part);
  else router_logits<DT, DT>(a, part);
}

// (registers: few enough that a block starts beside one of the first launch)
__global__ void __maxnreg__(160)
fp8_moe_kernel(const __grid_constant__ CUtensorMap t1, const __grid_constant__ CUtensorMap t2,
               const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap th,
               const __grid_constant__ Fp8MoeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Routes rt;
  __shared__ Phase phase[2];
  __shared__ Run run_slots[2];
  __shared__ int2 scan[kWarps];
  __shared__ uint32_t bits[kGateMaxExperts];
  Block b;
  b.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~static_cast<uintptr_t>(1023));
  b.base = smem_u32(b.smem);
  b.ctl = reinterpret_cast<CtaCtl*>(b.smem + kCtlOffset);
  b.status = a.status;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(b.smem + kCtlOffset + 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units1 = (a.I + 127) / 128, units2 = (a.N + 255) / 256;

  if (threadIdx.x == 0) {
    prefetch_map(&t1);
    prefetch_map(&t2);
    prefetch_map(&tx);
    prefetch_map(&th);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(b.full(s), 1);
      mbar_init(b.empty(s), 1);
    }
    for (int i = 0; i < kAccBufs; ++i) {
      mbar_init(b.accf(i), 2);                  // the sums, and the factors
      mbar_init(b.acce(i), 4);
    }
    mbar_init(b.drain(), 1);
    mbar_init(b.meet(), 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(b.run_given(i), 1);
      mbar_init(b.run_taken(i), kRunReaders);
    }
    mbar_init(b.chosen(), 1);
    b.ctl->abort = 0;
    b.ctl->timeout_ns = a.timeout_ns;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  auto set_phase = [&](int live) {
    if (warp == 0 && lane < 2)
      phase[lane].set(lane, ((lane ? a.I : a.K) + 127) / 128, lane ? units2 : units1, live);
  };
  // One token of the gate has topk distinct experts: all but their numbers and weights is known
  // now.  A warp without a role makes the choice while the others take up theirs, up to where
  // those are needed (phases, list and first steps between the choice and the first weights
  // otherwise: 64.5 -> 62.5 us).
  const bool one = a.T == 1 && a.router;
  if (one) {
    set_phase(a.rule.topk);
    if (warp == 3 && lane < a.rule.topk) {
      rt.start[lane] = rt.route[lane] = static_cast<int16_t>(lane);
      rt.tokens[lane] = 1u;
      if (lane == 0) rt.n_live = a.rule.topk;
    }
    __syncthreads();
  }
  grid_dependency_wait();
  uint32_t ticket = 0;
  if (threadIdx.x == 0) ticket = atomicAdd(a.counters, 1u);     // on its way meanwhile
  if (a.router) {
    const int t = one ? warp - 3 : warp;
    if (t >= 0 && t < a.T) {
      if (a.rule.E <= 128) gate_token<4>(a, rt, t);
      else if (a.rule.E <= 256) gate_token<8>(a, rt, t);
      else if (a.rule.E <= 512) gate_token<16>(a, rt, t);
      else gate_token<32>(a, rt, t);
      __syncwarp();
      if (one && lane == 0) mbar_arrive(b.chosen());
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
  if (!one) {
    __syncthreads();
    list_experts(a, rt, bits, scan);
    set_phase(rt.n_live);
    __syncthreads();
  }
  tc_fence_after();
  b.tmem = *tmem_slot;
  Runs runs{b, run_slots};
  Ring ring, acc;

  if (threadIdx.x == 0) {
    // -------------------------------------------------------------- producer
    const uint64_t wpol = l2_policy_evict_first(), tpol = l2_policy_evict_last();
    fence_proxy_async_global();                 // the codes of x were written before
    uint32_t issued = 0;
    bool alive = true, chosen = !one;
    int ph = 0;
#pragma unroll 1
    while (alive) {
      while (ph < 2 && ticket >= static_cast<uint32_t>(phase[ph].parts)) {
        ++ph;
        if (ph < 2) ticket = atomicAdd(a.counters + ph, 1u);
      }
      Run run{ph, static_cast<int>(ticket), 0, 0};
      if (ph < 2) {
        run.first = phase[ph].begin(run.number);
        run.count = phase[ph].begin(run.number + 1) - run.first;
      }
      if (!runs.give(run) || ph == 2) break;
      const Phase& p = phase[ph];
      const Producer copy{b, rt, p.down ? &t2 : &t1, p.down ? &th : &tx, wpol, tpol};
      // the weights of the first down tiles need no h
      const int early = p.down ? min(kStages, run.count) : 0;
      Ring ahead = ring;
      Cursor c;
      c.at(p, run.first);
#pragma unroll 1
      for (int i = -early; i < run.count; ++i) {
        if (i == 0 && early) {
          alive = wait_runs(a.counters + 2, static_cast<uint32_t>(phase[0].parts), b.ctl, b.status);
          if (!alive) break;
          fence_proxy_async_global();           // the codes of h
          c.at(p, run.first);
        }
        const bool weights = i < 0 || i >= early;
        Ring& at = i < 0 ? ahead : ring;
        if (weights) {
          if (!wait_soon(b.empty(at.slot), at.phase ^ 1u, b.ctl, b.status)) {
            alive = false;
            break;
          }
          if (!chosen) {
            alive = chosen = wait_soon(b.chosen(), 0, b.ctl, b.status);
            if (!alive) break;
          }
          copy.weights(p, c, at.slot);
          ++issued;
        }
        if (i >= 0) copy.tokens(p, c, at.slot);
        at.next(kStages);
        c.next(p);
      }
      if (alive) ticket = atomicAdd(a.counters + ph, 1u);
    }
    // what is on its way lands before the shared memory goes away
    const uint32_t late = issued > static_cast<uint32_t>(kStages) ? issued - kStages : 0u;
    for (uint32_t i = late; i < issued; ++i)
      wait_drain(b.full(static_cast<int>(i % kStages)), (i / kStages) & 1u,
                 b.ctl->timeout_ns);
  } else if (threadIdx.x == 32) {
    // ------------------------------------------------------------------- MMA
    const uint32_t idesc = idesc_e4m3(128, kCols);
    bool alive = true;
    Run run;
#pragma unroll 1
    while (alive && runs.take(&run, false) && run.phase < 2) {
#pragma unroll 1
      for (int i = 0; i < run.count; ++i) {
        if (!wait_both(b.acce(acc.slot), acc.phase ^ 1u, b.full(ring.slot), ring.phase, b.ctl,
                       b.status)) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint32_t s = b.stage(ring.slot), d = b.tmem + acc.slot * 2 * kCols;
        const uint64_t tok = sdesc_sw128(s + kTokOffset);
        tc_mma_e4m3_k128(d, sdesc_sw128(s), tok, idesc);
        tc_mma_e4m3_k128(d + kCols, sdesc_sw128(s + kGroupBytes), tok, idesc);
        tc_commit(b.accf(acc.slot));
        tc_commit(b.empty(ring.slot));
        ring.next(kStages);
        acc.next(kAccBufs);
      }
    }
    tc_commit(b.drain());
    wait_drain(b.drain(), 0, b.ctl->timeout_ns);
  } else if (warp == 2) {
    Run run;
    const bool ready =
        !one || __all_sync(kFullWarp, wait_soon(b.chosen(), 0, b.ctl, b.status));
    while (ready && runs.take(&run, true) && run.phase < 2) {
      if (run.phase == 1) {                     // the scales of h
        bool ok = true;
        if (lane == 0)
          ok = wait_runs(a.counters + 2, static_cast<uint32_t>(phase[0].parts), b.ctl, b.status);
        if (!__all_sync(kFullWarp, ok)) break;
      }
      factors(b, a, rt, phase[run.phase], run, acc);
    }
  } else if (warp >= 4) {
    Epilogue epi{b, a, rt, static_cast<int>(threadIdx.x) & 127};
    Run run;
    bool warm = true;
    while (runs.take(&run, true) && run.phase < 2) {
      if (!epi.add(phase[run.phase], run, acc, warm && run.phase == 0)) break;
      warm = false;
    }
  }
  __syncwarp();
  if (rt.n_live == 0)                           // no route at all
    for (int64_t i = blockIdx.x * kThreads + threadIdx.x; i < static_cast<int64_t>(a.T) * a.N;
         i += static_cast<int64_t>(gridDim.x) * kThreads)
      static_cast<uint16_t*>(a.out)[i / a.N * a.ldo + i % a.N] = 0;
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(b.tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t init_fp8_moe_attributes() {
  cudaError_t e = cudaFuncSetAttribute(fp8_moe_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmemBytes);
  // The first launch has the SM's memory split as the second needs it: a block of that can
  // then start beside one of this (with another split it starts when the SM is empty).
  for (auto* f : {fp8_moe_router_kernel<NVFP4_BF16>, fp8_moe_router_kernel<NVFP4_FP16>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
  return e;
}

int fp8_moe_box_rows() { return kCols; }

bool fp8_moe_layout(int64_t T, int32_t topk, int32_t E, int64_t K, int64_t I, int64_t N,
                    MoeLayout* m) {
  if (T <= 0 || topk <= 0 || E <= 0 || topk > E || K <= 0 || I <= 0 || N <= 0 || K % 16 != 0 ||
      I % 16 != 0 || T > kMoeMaxTokens || T * topk > kMoeMaxRoutes || E > kGateMaxExperts ||
      topk > kGateMaxTopk || K > (1 << 20) || I > (1 << 20) || N > (1 << 20))
    return false;
  const int64_t R = T * topk;
  const int64_t live = R < E ? R : E, kx = (K + 127) / 128, kh = (I + 127) / 128;
  const int64_t units2 = (N + 255) / 256;
  // tiles times blocks stay below 2^32
  if (live * kh * (kx > units2 ? kx : units2) > 0xFFFFFFFFLL / kMoeMaxGrid - 1) return false;
  size_t end = 0;
  auto take = [&](int64_t bytes) {
    const size_t at = end;
    end += static_cast<size_t>((bytes + 255) / 256 * 256);
    return at;
  };
  m->columns = TB;
  m->experts = static_cast<int>(live);
  m->ld_xq = kx * 128;
  m->ld_hq = kh * 128;
  take(T * E * 4);
  m->xq = take(m->columns * m->ld_xq);
  m->xs = take(kx * m->columns * 4);
  // (one expert more: what Epilogue::add warms up on)
  m->hq = take((live + 1) * m->columns * m->ld_hq);
  m->hs = take((live + 1) * kh * m->columns * 4);
  m->part = take(static_cast<int64_t>(2) * kMoeMaxGrid * 2 * m->columns * 128 * 4);
  m->counters = take((4 + live * kh + 4 * units2) * 4);
  m->bytes = end;
  return true;
}

cudaError_t launch_fp8_moe(const CUtensorMap& t1, const CUtensorMap& t2, const CUtensorMap& tx,
                           const CUtensorMap& th, const Fp8MoeArgs& a, int sms, cudaStream_t s) {
  const int grid = sms < kMoeMaxGrid ? sms : kMoeMaxGrid;
  // one or two blocks an SM: a row and four tokens each, as far as that goes
  const int first = a.router && a.rule.E * ((a.T + 3) / 4) > grid ? 2 * grid : grid;
  if (a.type == NVFP4_BF16) fp8_moe_router_kernel<NVFP4_BF16><<<first, kThreads, 0, s>>>(a);
  else fp8_moe_router_kernel<NVFP4_FP16><<<first, kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, fp8_moe_kernel, t1, t2, tx, th, a);
}

}  // namespace nvfp4
