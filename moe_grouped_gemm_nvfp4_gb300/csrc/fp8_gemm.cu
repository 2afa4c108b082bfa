// FP8 block-scaled GEMM, weight rows on the MMA's M side: one tile is 128
// weight rows (one 128 x 128 scale block high) x NT tokens, dense or grouped
// by expert.
//
//   y[m, n] = sum_b sa[m, b] sw[n / 128, b] sum_{k in block b} qa[m, k] qw[n, k]
//
// The inner sum of one K block (four K = 32 MMAs) is the only part the tensor
// cores can add up by themselves: the scales are FP32 and change with b.  So
// every K block gets an accumulator of its own in a ring of tensor-memory
// buffers, and the epilogue warps add it, times sa * sw, into FP32 registers
// while the next blocks' MMAs run.  A thread holds one weight row and NT (or
// NT / 2) tokens, so the factors are per column: one warp writes the NT
// products sa * sw of each K block to shared memory, where the epilogue reads
// them as broadcasts.
//
// Roles (one persistent CTA per SM): warp 0 TMA producer (weights 16 KB and
// NT rows of activations per stage), warp 1 tensor memory and MMA, warp 2
// factors, warp 3 zeros the output rows past the last expert's, warps 4..
// epilogue (4, or 8 for NT = 128).  Few units and a long
// K: the CTAs of a cluster share a unit, each a slice of K, and sum their
// registers through distributed shared memory in rank order (no atomics, the
// same bits every time).  Every wait is bounded.
#include "fp8_common.cuh"

namespace nvfp4 {

namespace {

constexpr int kWBytes = 128 * 128;           // one weight tile of a K block

template <int NT>
struct Cfg {
  static constexpr int kABytes = NT * 128;
  static constexpr int kStageBytes = kWBytes + kABytes;
  static constexpr int kStages = NT <= 32 ? 10 : (NT == 64 ? 8 : 6);
  static constexpr int kBufs = 4;            // accumulators in flight
  static constexpr int kTmemCols = NT * kBufs;
  static constexpr int kEpiWarps = NT == 128 ? 8 : 4;
  static constexpr int kCols = NT == 128 ? 64 : NT;      // columns a thread holds
  static constexpr int kThreads = 128 + 32 * kEpiWarps;
  static constexpr int kUnitBytes = 2 * 4 * (kFp8MaxExperts + 1) + 8;
  static constexpr int kFacOffset = kStages * kStageBytes;
  static constexpr int kUnitOffset = kFacOffset + kBufs * NT * 4;
  static constexpr int kBarOffset = (kUnitOffset + kUnitBytes + 7) / 8 * 8;
  // full[S], empty[S], acc_full[B], acc_empty[B], fac_full[B], drain
  static constexpr int kBarBytes = 8 * (2 * kStages + 3 * kBufs + 1);
  static constexpr int kCtlOffset = kBarOffset + kBarBytes;
  static constexpr int kSmemBytes = kCtlOffset + 64 + 1024;   // + alignment slack
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert(NT * 128 * 4 <= kStages * kStageBytes, "the K-split sums reuse the stages");
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "");
};

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void store_out(const Fp8GemmArgs& a, int row, int n, float v) {
  const int64_t at = static_cast<int64_t>(row) * a.ldc + n;
  if (a.out_type == NVFP4_FP32) static_cast<float*>(a.out)[at] = v;
  else static_cast<uint16_t*>(a.out)[at] = f32_to_out16(v, a.out_type);
}

// SPLIT: one unit per cluster, K shared by its CTAs; otherwise persistent.
template <int NT, bool SPLIT>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tw,
                const Fp8GemmArgs a) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBarOffset;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::kStages + s); };
  auto accf_bar = [&](int b) { return bar0 + 8u * (2 * C::kStages + b); };
  auto acce_bar = [&](int b) { return bar0 + 8u * (2 * C::kStages + C::kBufs + b); };
  auto facf_bar = [&](int b) { return bar0 + 8u * (2 * C::kStages + 2 * C::kBufs + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * C::kStages + 3 * C::kBufs);
  CtaCtl* ctl = reinterpret_cast<CtaCtl*>(smem + C::kCtlOffset);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kCtlOffset + 16);
  float* fac = reinterpret_cast<float*>(smem + C::kFacOffset);
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
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), C::kEpiWarps);
      mbar_init(facf_bar(b), 1);
    }
    mbar_init(drain_bar, 1);
    ctl->abort = 0;
    ctl->timeout_ns = a.timeout_ns;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
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
  uint32_t issued = 0;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // weights pass through once unless several token tiles share them
    const uint64_t wpol = l2_policy_evict_first();
    const uint64_t apol = l2_policy_evict_last();
    int stage = 0;
    uint32_t phase = 0;
    bool alive = true;
    for (int u = u0; u < units && alive; u += ustep) {
      const Unit un = unit_at(um, u);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(empty_bar(stage), phase ^ 1u, ctl, a.status))) {
          alive = false;
          break;
        }
        if (!((a.debug_flags & kFp8SkipFirstStage) && issued == 0)) {
          const uint32_t dst = sbase + stage * C::kStageBytes;
          mbar_arrive_expect_tx_elect(full_bar(stage), C::kStageBytes);
          tma_load_3d_elect(dst, &tw, full_bar(stage), kb * 128, un.nt * 128, un.e, wpol);
          tma_load_2d_elect(dst + kWBytes, &ta, full_bar(stage), kb * 128, un.row, apol);
        }
        ++issued;
        if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    const uint32_t idesc = idesc_e4m3(128, NT);
    int stage = 0, buf = 0;
    uint32_t phase = 0, bphase = 0;
    bool alive = true;
    for (int u = u0; u < units && alive; u += ustep) {
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(acce_bar(buf), bphase ^ 1u, ctl, a.status) &&
                                         mbar_wait(full_bar(stage), phase, ctl, a.status))) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint32_t src = sbase + stage * C::kStageBytes;
        const uint64_t dw = sdesc_sw128(src);
        const uint64_t da = sdesc_sw128(src + kWBytes);
        // columns past K arrive as zeros
        const int ksteps = min(4, (a.K - kb * 128 + 31) >> 5);
        for (int ks = 0; ks < ksteps; ++ks)
          tc_mma_e4m3_elect(tmem + buf * NT, dw + 2 * ks, da + 2 * ks, idesc, ks > 0 ? 1u : 0u);
        tc_commit_elect(empty_bar(stage));
        tc_commit_elect(accf_bar(buf));
        if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
        if (++buf == C::kBufs) { buf = 0; bphase ^= 1u; }
      }
    }
    tc_commit_elect(drain_bar);
    if (lane == 0) wait_drain(drain_bar, 0, ctl->timeout_ns);
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------- factors
    constexpr int kPer = (NT + 31) / 32;      // tokens per lane
    constexpr int kAhead = 4;                 // K blocks loaded ahead
    int buf = 0;
    uint32_t bphase = 0;
    bool alive = true;
    for (int u = u0; u < units && alive; u += ustep) {
      const Unit un = unit_at(um, u);
      const float* sw = a.sw + (static_cast<int64_t>(un.e) * a.nnb + un.nt) * a.nkb;
      float na[kAhead][kPer], nw[kAhead];
      auto fetch = [&](int kb) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const bool in = kb + j < kb1;
          nw[j] = in ? __ldg(sw + kb + j) : 0.f;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int col = lane + 32 * i;
            na[j][i] = in && col < un.cnt ? __ldg(a.sa + (kb + j) * a.lds + un.row + col) : 0.f;
          }
        }
      };
      fetch(kb0);
      for (int kb = kb0; kb < kb1 && alive; kb += kAhead) {
        float f[kAhead][kPer];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
          for (int i = 0; i < kPer; ++i) f[j][i] = na[j][i] * nw[j];
        fetch(kb + kAhead);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (kb + j >= kb1 || !alive) break;
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(acce_bar(buf), bphase ^ 1u, ctl, a.status))) {
            alive = false;
            break;
          }
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < NT) fac[buf * NT + lane + 32 * i] = f[j][i];
          __syncwarp();
          if (lane == 0) mbar_arrive(facf_bar(buf));
          if (++buf == C::kBufs) { buf = 0; bphase ^= 1u; }
        }
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------- rows of no expert are zero
    if (um.first) zero_rows_past(a, um.first[a.E], lane);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                        // tensor-memory lane quarter
    const int c0 = ((warp - 4) >> 2) * C::kCols;   // first column of this group
    int buf = 0;
    uint32_t bphase = 0;
    bool alive = true;
    for (int u = u0; u < units && alive; u += ustep) {
      float acc[C::kCols];
#pragma unroll
      for (int i = 0; i < C::kCols; ++i) acc[i] = 0.f;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(facf_bar(buf), bphase, ctl, a.status) &&
                                         mbar_wait(accf_bar(buf), bphase, ctl, a.status))) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * NT + c0;
        const float4* fp = reinterpret_cast<const float4*>(fac + buf * NT + c0);
        constexpr int kChunk = C::kCols < 32 ? C::kCols : 32;
#pragma unroll
        for (int h = 0; h < C::kCols / kChunk; ++h) {
          uint32_t r[kChunk];
          if constexpr (kChunk == 16) tmem_ld16(taddr, r);
          else tmem_ld32(taddr + h * 32, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < kChunk / 4; ++i) {
            const float4 f = fp[h * (kChunk / 4) + i];
            float* d = acc + h * kChunk + 4 * i;
            fma_pair(d[0], d[1], r[4 * i], r[4 * i + 1], f.x, f.y);
            fma_pair(d[2], d[3], r[4 * i + 2], r[4 * i + 3], f.z, f.w);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acce_bar(buf));
        if (++buf == C::kBufs) { buf = 0; bphase ^= 1u; }
      }
      if (!alive) break;
      if constexpr (SPLIT) {
        // every MMA and copy of this CTA has completed: the stages are free
        float* red = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int i = 0; i < C::kCols; ++i) red[(c0 + i) * 128 + q * 32 + lane] = acc[i];
      } else {
        const Unit un = unit_at(um, u);
        const int n = un.nt * 128 + q * 32 + lane;
        if (n < a.N) {
#pragma unroll
          for (int i = 0; i < C::kCols; ++i)
            if (c0 + i < un.cnt) store_out(a, un.row + c0 + i, n, acc[i]);
        }
      }
    }
  }

  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync_all();
    if (u0 < units) {
      // each CTA adds up the ranks' sums of its share of the columns
      const Unit un = unit_at(um, u0);
      const int n = threadIdx.x & 127;
      for (int c = rank + nsplit * static_cast<int>(threadIdx.x >> 7); c < un.cnt;
           c += nsplit * (C::kThreads / 128)) {
        float v = 0.f;
        for (int j = 0; j < nsplit; ++j)
          v += ld_cluster_f32(mapa_shared(sbase + (c * 128 + n) * 4, j));
        if (un.nt * 128 + n < a.N) store_out(a, un.row + c, un.nt * 128 + n, v);
      }
    }
    cluster_sync_all();
  }

  // Teardown: the copies still in flight (after an abort) land before the
  // shared memory goes away; the MMAs have drained in warp 1.
  tc_fence_before();
  __syncthreads();
  if (warp == 0 && lane == 0) {
    const uint32_t from = issued > static_cast<uint32_t>(C::kStages) ? issued - C::kStages : 0u;
    const uint32_t skip = (a.debug_flags & kFp8SkipFirstStage) ? 1u : 0u;
    for (uint32_t i = from; i < issued; ++i)
      if (i >= skip)
        wait_drain(full_bar(static_cast<int>(i % C::kStages)), (i / C::kStages) & 1u,
                   ctl->timeout_ns);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int NT, bool SPLIT>
cudaError_t set_attr() {
  cudaError_t e = cudaFuncSetAttribute(fp8_gemm_kernel<NT, SPLIT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<NT>::kSmemBytes);
  return e;
}

template <int NT>
cudaError_t launch(const CUtensorMap& ta, const CUtensorMap& tw, const Fp8GemmArgs& a, int sms,
                   cudaStream_t s) {
  const int64_t ntiles = (a.N + 127) / 128;
  // upper bound of the token tiles
  const int64_t some = a.offsets ? (a.rows < a.E ? a.rows : a.E) : 1;
  const int64_t ttiles = a.offsets ? some + (a.rows - some) / NT : (a.rows + NT - 1) / NT;
  const int64_t units = ntiles * ttiles;
  if (units > 0x3FFFFFFF) return cudaErrorInvalidConfiguration;
  // K over the CTAs of a cluster while two of them per unit still fit the GPU
  int split = 1;
  while (split < 8 && units * split * 2 <= sms && a.nkb >= 4 * split) split *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(Cfg<NT>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg<NT>::kSmemBytes;
  cfg.stream = s;
  if (split == 1) {
    cfg.gridDim = dim3(static_cast<unsigned>(units < sms ? units : sms), 1, 1);
    return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<NT, false>, ta, tw, a);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(units * split), 1, 1);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<NT, true>, ta, tw, a);
}

}  // namespace

cudaError_t init_fp8_gemm_attributes() {
  cudaError_t e = cudaSuccess;
  if (e == cudaSuccess) e = set_attr<16, false>();
  if (e == cudaSuccess) e = set_attr<32, false>();
  if (e == cudaSuccess) e = set_attr<64, false>();
  if (e == cudaSuccess) e = set_attr<128, false>();
  if (e == cudaSuccess) e = set_attr<16, true>();
  if (e == cudaSuccess) e = set_attr<32, true>();
  if (e == cudaSuccess) e = set_attr<64, true>();
  if (e == cudaSuccess) e = set_attr<128, true>();
  return e;
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
