// FP8 block-scaled GEMM, one CTA per tile of up to 128 tokens x 128 weight rows
// (one 128 x 128 scale block high), dense or grouped by expert.
//
//   y[m, n] = sum_b sa[m, b] sw[n / 128, b] sum_{k in block b} qa[m, k] qw[n, k]
//
// The inner sum of one K block (four K = 32 MMAs) is the only part the tensor
// cores can add up by themselves: the scales are FP32 and change with b.  So
// every K block gets an accumulator of its own in a ring of four tensor-memory
// buffers, and the epilogue warps add it, times sa * sw, into FP32 registers
// while the next blocks' MMAs run.  The tokens are the accumulator's rows: a
// thread holds one token and 64 weight rows of one scale block, so its factor
// is one value per K block.  (With the weights as rows the factors differ by
// column; reading them from shared memory, 128 per K block and lane quarter,
// took 512 of the LSU's cycles per 256-cycle K block.)  The MMA always spans
// 128 rows; with fewer tokens per tile (NT) only their rows are loaded, the
// rest of the operand is the stage's weights, and those accumulator rows are
// never read.  Weights stream at the HBM rate long before the MMA's 256 cycles
// per 16 KB matter (a K block's weights take about 700).
//
// Roles (one persistent CTA per SM): warp 0 TMA producer (weights 16 KB and
// NT rows of activations per stage), warp 1 tensor memory and MMA, warp 2 the
// factors (shared memory, one set per accumulator buffer; its arrival counts
// on the buffer's barrier beside the MMA's), warp 3 zeros the output rows past
// the last expert's, warps 4-11 epilogue (lane quarter warp % 4, 64 columns
// each).  Few units and a long K: the CTAs of a cluster share a unit, each a
// slice of K, and sum their registers through distributed shared memory in rank
// order (no atomics, the same bits every time).  Every wait is bounded.
//
// Measured with the quantiser: 128 experts' gate_up at 16 tokens each 461 us (3.2
// GB of weights at 7.0 TB/s; a copy moves 6.8), down at 64 tokens 262 us (6.7 TB/s),
// 8192^3 467 us (2.35 PFLOP/s, 0.63 of twice the BF16 rate), 4096 x 4096 x 6144 97 us, the
// skewed 65536-route prefill 1.82 ms.  Many tokens are bound by two things at once,
// both per K block: the way through MMA warp, accumulator, epilogue and back
// (about 430 cycles with the ring full; 355 without loads, reads and additions)
// and the 32 KB that come in from L2 (66 bytes a cycle and SM).  Under load the
// board's power limit takes the clock from 1.95 to 1.67 GHz (prefill 1.51).  Tried:
// CTA pairs of 256 x 256 (two accumulators; 133 us where this took 98), 256 x 128
// (124), one CTA of 128 x 256 with 16 epilogue warps (138).
#include "fp8_common.cuh"

namespace nvfp4 {

namespace {

constexpr int kWBytes = 128 * 128;           // one weight tile of a K block

template <int NT>
struct Cfg {
  static constexpr int kABytes = NT * 128;
  static constexpr int kStageBytes = kABytes + kWBytes;   // A first: see load_a
  static constexpr int kStages = NT <= 32 ? 10 : (NT == 64 ? 8 : 6);
  static constexpr int kBufs = 4;            // accumulators in flight
  static constexpr int kQuarters = (NT + 31) / 32;
  static constexpr int kCols = 64;           // columns a thread holds
  static constexpr int kThreads = 128 + 256;
  static constexpr int kUnitBytes = 2 * 4 * (kFp8MaxExperts + 1) + 8;
  static constexpr int kFacOffset = kStages * kStageBytes;
  // rows on their way out, one buffer per epilogue warp
  static constexpr int kStoreOffset = kFacOffset + kBufs * 128 * 4;
  static constexpr int kUnitOffset = kStoreOffset + 2 * kQuarters * kStoreWords * 4;
  static constexpr int kBarOffset = (kUnitOffset + kUnitBytes + 7) / 8 * 8;
  // full[S], empty[S], acc_full[B], acc_empty[B], drain
  static constexpr int kBarBytes = 8 * (2 * kStages + 2 * kBufs + 1);
  static constexpr int kCtlOffset = kBarOffset + kBarBytes;
  static constexpr int kSmemBytes = kCtlOffset + 64 + 1024;   // + alignment slack
  // K-split sums: a row of 128 columns per token, four words of padding (rows of
  // neighbouring lanes then lie in different banks for 16-byte accesses)
  static constexpr int kRedStride = 132;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert(NT * kRedStride * 4 <= kStages * kStageBytes, "the K-split sums reuse the stages");
};

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// Four neighbouring outputs of one row (those before column N).
__device__ __forceinline__ void store_four(const Fp8GemmArgs& a, int row, int n, const float4& v) {
  const int64_t at = static_cast<int64_t>(row) * a.ldc + n;
  const float f[4] = {v.x, v.y, v.z, v.w};
  if (a.out_type == NVFP4_FP32) {
    float* dst = static_cast<float*>(a.out) + at;
    if (a.vec && n + 4 <= a.N) {
      *reinterpret_cast<float4*>(dst) = v;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < a.N) dst[j] = f[j];
    }
  } else {
    uint16_t* dst = static_cast<uint16_t*>(a.out) + at;
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = f32_to_out16(f[j], a.out_type);
    if (a.vec && n + 4 <= a.N) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < a.N) dst[j] = static_cast<uint16_t>(h[j]);
    }
  }
}

// kSplit: one unit per cluster, K shared by its CTAs.  Persistent otherwise, with
// outputs in rows of 16-byte chunks or in any.
enum Mode : int { kChunkRows, kAnyRows, kSplit };
template <int NT, int MODE>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tw,
                const Fp8GemmArgs a) {
  using C = Cfg<NT>;
  constexpr bool SPLIT = MODE == kSplit;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBarOffset;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::kStages + s); };
  auto accf_bar = [&](int b) { return bar0 + 8u * (2 * C::kStages + b); };
  auto acce_bar = [&](int b) { return bar0 + 8u * (2 * C::kStages + C::kBufs + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * C::kStages + 2 * C::kBufs);
  const uint32_t fac = sbase + C::kFacOffset;
  CtaCtl* ctl = reinterpret_cast<CtaCtl*>(smem + C::kCtlOffset);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kCtlOffset + 16);
  int* first = reinterpret_cast<int*>(smem + C::kUnitOffset);
  int* tiles = first + kFp8MaxExperts + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(accf_bar(b), 2);                 // the sums, and the factors
      mbar_init(acce_bar(b), 128 / C::kCols * C::kQuarters);
    }
    mbar_init(drain_bar, 1);
    ctl->abort = 0;
    ctl->timeout_ns = a.timeout_ns;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (a.offsets) load_units(a.offsets, a.E, a.rows, NT, first, tiles, a.status);
  UnitMap um;
  um.first = a.offsets ? first : nullptr;
  um.tiles = tiles;
  um.E = a.E;
  um.rows = a.rows;
  um.ntiles = (a.N + 127) >> 7;
  um.ttiles = (a.rows + NT - 1) / NT;
  um.width = NT;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int units = unit_count(um);
  const int nsplit = SPLIT ? static_cast<int>(cluster_nctarank()) : 1;
  const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  const int u0 = static_cast<int>(blockIdx.x) / nsplit;
  const int ustep = SPLIT ? units + 1 : static_cast<int>(gridDim.x);   // SPLIT: one unit
  const int kb0 = SPLIT ? a.nkb * rank / nsplit : 0;
  const int kb1 = SPLIT ? a.nkb * (rank + 1) / nsplit : a.nkb;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      uint32_t issued = 0;
      // Weights: out of L2 first, so that the activations stay (one tile of tokens
      // per expert reads them once; 4096 x 4096 x 6144 97.6 us, 106.1 us kept like
      // other lines), except where experts have several tiles of tokens that share
      // them in passing (64 experts, 16384 routes, N 3000, K 4096: 298 and 267 us;
      // the 65536-route prefill 2.04 and 1.88 ms).  Rows that start inside a
      // 128-byte line go out first there too (K 4080: 334 and 385 us).
      const bool shared_w = NT == 128 && a.offsets != nullptr && (a.K & 127) == 0;
      const uint64_t wpol = shared_w ? l2_policy_evict_normal() : l2_policy_evict_first();
      const uint64_t apol = l2_policy_evict_last();
      auto load_w = [&](const Unit& un, int kb, int s) {
        mbar_arrive_expect_tx(full_bar(s), C::kStageBytes);
        tma_load_3d(sbase + s * C::kStageBytes + C::kABytes, &tw, full_bar(s), kb * 128,
                    un.nt * 128, un.e, wpol);
      };
      // NT rows; the MMA reads 128 from here: the rest are the weights after them
      auto load_a = [&](const Unit& un, int kb, int s) {
        tma_load_2d(sbase + s * C::kStageBytes, &ta, full_bar(s), kb * 128, un.row, apol);
      };
      const bool skip = (a.debug_flags & kFp8SkipFirstStage) != 0;
      int stage = 0;
      uint32_t phase = 0;
      bool alive = true;
      // The weights of the first stages need nothing from the kernel before
      // (the activations' quantiser, when this one was launched to overlap it).
      const int ahead = u0 < units ? min(C::kStages, kb1 - kb0) : 0;
      if (ahead > 0) {
        const Unit un = unit_at(um, u0);
        for (int i = 0; i < ahead; ++i)
          if (!(skip && i == 0)) load_w(un, kb0 + i, i);
        grid_dependency_wait();
        for (int i = 0; i < ahead; ++i)
          if (!(skip && i == 0)) load_a(un, kb0 + i, i);
        issued = ahead;
        stage = ahead == C::kStages ? 0 : ahead;
        phase = ahead == C::kStages ? 1u : 0u;
      }
      int from = kb0 + ahead;
      for (int u = u0; u < units && alive; u += ustep) {
        const Unit un = unit_at(um, u);
        for (int kb = from; kb < kb1; ++kb) {
          if (!wait_soon(empty_bar(stage), phase ^ 1u, ctl, a.status)) {
            alive = false;
            break;
          }
          load_w(un, kb, stage);
          load_a(un, kb, stage);
          ++issued;
          if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
        }
        from = kb0;
      }
      // Copies still in flight after an abort land before the shared memory
      // goes away (complete already otherwise).
      const uint32_t late = issued > static_cast<uint32_t>(C::kStages) ? issued - C::kStages : 0u;
      for (uint32_t i = late; i < issued; ++i)
        if (!(skip && i == 0))
          wait_drain(full_bar(static_cast<int>(i % C::kStages)), (i / C::kStages) & 1u,
                     ctl->timeout_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    if (elect_one()) {
      const uint32_t idesc = idesc_e4m3(128, 128);
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      bool alive = true;
      for (int u = u0; u < units && alive; u += ustep) {
        for (int kb = kb0; kb < kb1; ++kb) {
          const uint32_t src = sbase + stage * C::kStageBytes;
          if (!wait_both(acce_bar(buf), bphase ^ 1u, full_bar(stage), phase, ctl, a.status)) {
            alive = false;
            break;
          }
          tc_fence_after();
          tc_mma_e4m3_k128(tmem + buf * 128, sdesc_sw128(src), sdesc_sw128(src + C::kABytes),
                           idesc);
          tc_commit(accf_bar(buf));
          tc_commit(empty_bar(stage));
          if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
          if (++buf == C::kBufs) { buf = 0; bphase ^= 1u; }
        }
      }
      tc_commit(drain_bar);
      wait_drain(drain_bar, 0, ctl->timeout_ns);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------- factors
    grid_dependency_wait();
    factor_units<NT, C::kBufs>(
        a, um, u0, units, ustep, kb0, kb1, fac, lane,
        [&](int b, uint32_t phase) {
          return __all_sync(0xFFFFFFFFu, wait_soon(acce_bar(b), phase ^ 1u, ctl, a.status)) != 0;
        },
        [&](int b) { mbar_arrive(accf_bar(b)); });
  } else if (warp == 3) {
    // ------------------------------------------- rows of no expert are zero
    if (um.first) zero_rows_past(a, um.first[a.E], lane);
  } else if (warp >= 4 && (warp & 3) < C::kQuarters) {
    // ------------------------------------------------------------ epilogue
    const int row = (warp & 3) * 32 + lane;        // token within the tile
    const int c0 = ((warp - 4) >> 2) * C::kCols;   // first column of this group
    const uint32_t tbase = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0;
    int buf = 0;
    uint32_t bphase = 0;
    for (int u = u0; u < units; u += ustep) {
      const Unit un = unit_at(um, u);
      uint64_t acc[C::kCols / 2];
#pragma unroll
      for (int i = 0; i < C::kCols / 2; ++i) acc[i] = 0;
      const bool alive = add_unit<C::kCols, C::kBufs>(
          acc, kb1 - kb0, tbase, buf, bphase,
          [&](int b, uint32_t phase) {
            const bool ok = __all_sync(0xFFFFFFFFu, wait_soon(accf_bar(b), phase, ctl, a.status));
            tc_fence_after();
            return ok;
          },
          [&](int b) { return ld_shared_f32(fac + 4 * (b * 128 + row)); },
          [&](int b) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acce_bar(b));
          });
      if (!alive) break;
      if constexpr (SPLIT) {
        // every MMA and copy of this CTA has completed: the stages are free
        if (row < NT) {
          float4* red =
              reinterpret_cast<float4*>(smem + 4 * (row * C::kRedStride + c0));
#pragma unroll
          for (int i = 0; i < C::kCols / 4; ++i) {
            float4 v;
            unpack2(acc[2 * i], v.x, v.y);
            unpack2(acc[2 * i + 1], v.z, v.w);
            red[i] = v;
          }
        }
      } else {
        const int q = warp & 3;
        store_rows<C::kCols, MODE == kChunkRows>(
            a, un.row + 32 * q, un.cnt - 32 * q, un.nt * 128 + c0, acc,
            sbase + C::kStoreOffset + 4 * kStoreWords * (((warp - 4) >> 2) * C::kQuarters + q),
            lane);
      }
    }
  }

  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync_all();
    if (u0 < units) {
      // each CTA adds up the ranks' sums of its share of the tokens, four columns
      // a thread; the reads of other CTAs take long, so those of two tokens and
      // all ranks are in flight together
      const Unit un = unit_at(um, u0);
      const int n = 4 * (threadIdx.x & 31);
      constexpr int kGroups = C::kThreads / 32;
      constexpr int kTogether = 2, kRanks = 8;
      const int step = nsplit * kGroups;
      for (int t0 = rank + nsplit * static_cast<int>(threadIdx.x >> 5); t0 < un.cnt;
           t0 += kTogether * step) {
        float4 v[kTogether][kRanks];
#pragma unroll
        for (int i = 0; i < kTogether; ++i)
#pragma unroll
          for (int j = 0; j < kRanks; ++j)
            v[i][j] = j < nsplit && t0 + i * step < un.cnt
                          ? ld_cluster_f4(mapa_shared(
                                sbase + 4 * ((t0 + i * step) * C::kRedStride + n), j))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
          if (t0 + i * step >= un.cnt) break;
          float4 o = v[i][0];
#pragma unroll
          for (int j = 1; j < kRanks; ++j) {
            o.x += v[i][j].x; o.y += v[i][j].y; o.z += v[i][j].z; o.w += v[i][j].w;
          }
          const int row = un.row + t0 + i * step, col = un.nt * 128 + n;
          store_four(a, row, col, o);
        }
      }
    }
    cluster_sync_all();
  }

  // The producer's copies have landed and the MMAs have drained.
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int NT, int MODE>
cudaError_t set_attr() {
  return cudaFuncSetAttribute(fp8_gemm_kernel<NT, MODE>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<NT>::kSmemBytes);
}

template <int NT>
cudaError_t set_attrs() {
  cudaError_t e = set_attr<NT, kChunkRows>();
  if (e == cudaSuccess) e = set_attr<NT, kAnyRows>();
  return e == cudaSuccess ? set_attr<NT, kSplit>() : e;
}

template <int NT>
cudaError_t launch(const CUtensorMap& ta, const CUtensorMap& tw, const Fp8GemmArgs& a, int sms,
                   cudaStream_t s) {
  using C = Cfg<NT>;
  // upper bound of the token tiles
  const int64_t some = a.offsets ? (a.rows < a.E ? a.rows : a.E) : 1;
  const int64_t ttiles = a.offsets ? some + (a.rows - some) / NT : (a.rows + NT - 1) / NT;
  const int64_t units = (a.N + 127) / 128 * ttiles;
  if (units > 0x3FFFFFFF) return cudaErrorInvalidConfiguration;
  // K over the CTAs of a cluster while two of them per unit still fit the GPU
  int split = 1;
  while (split < 8 && units * split * 2 <= sms && a.nkb >= 4 * split) split *= 2;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  if (a.overlap) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (split == 1) {
    cfg.gridDim = dim3(static_cast<unsigned>(units < sms ? units : sms), 1, 1);
    return a.vec ? cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<NT, kChunkRows>, ta, tw, a)
                 : cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<NT, kAnyRows>, ta, tw, a);
  }
  attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
  attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(split);
  attr[cfg.numAttrs].val.clusterDim.y = 1;
  attr[cfg.numAttrs++].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(units * split), 1, 1);
  return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<NT, kSplit>, ta, tw, a);
}

}  // namespace

cudaError_t init_fp8_gemm_attributes() {
  cudaError_t e = set_attrs<16>();
  if (e == cudaSuccess) e = set_attrs<32>();
  if (e == cudaSuccess) e = set_attrs<64>();
  return e == cudaSuccess ? set_attrs<128>() : e;
}

// Tokens per tile: the rows themselves for one matrix; for E experts 1.6
// times the mean, so that an expert of a balanced routing fits one tile and
// its weights are read once.
int fp8_tile_tokens(int64_t rows, int32_t E) {
  const int64_t want = E > 0 ? (rows * 8 + E * 5LL - 1) / (E * 5LL) : rows;
  return want <= 16 ? 16 : want <= 32 ? 32 : want <= 80 ? 64 : 128;
}

cudaError_t launch_fp8_gemm(const CUtensorMap& ta, const CUtensorMap& tw, const Fp8GemmArgs& a,
                            int sms, cudaStream_t s) {
  switch (fp8_tile_tokens(a.rows, a.offsets ? a.E : 0)) {
    case 16: return launch<16>(ta, tw, a, sms, s);
    case 32: return launch<32>(ta, tw, a, sms, s);
    case 64: return launch<64>(ta, tw, a, sms, s);
    default: return launch<128>(ta, tw, a, sms, s);
  }
}

}  // namespace nvfp4
