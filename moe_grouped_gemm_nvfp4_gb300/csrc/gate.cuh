// The top-k gate of one token by one warp: scores, choice and weights.
//
//   s = softmax(l) or 1 / (1 + exp(-l));  chosen: the topk largest l, or, with a bias,
//   s + bias, best first, the lower number first among equals;  w = s of the chosen
//   [/ their sum] * scale
//
// Lane i of the warp holds the experts i, i + 32, ...: a choice is a maximum of
// order-preserving integers over the lane's own, then over the lanes (an integer
// reduction, a vote for who has it, among equals another for the lowest number).  A NaN
// counts as the largest value.  With a bias the chosen order hangs on sums whose 32-bit rounding
// can swap neighbours; where two neighbours of the order (the first one left out
// among them) are nearer than that rounding, the token is chosen again on 64-bit
// keys.  64-bit exponentials for all would take longer than everything else here.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "common.cuh"

namespace nvfp4 {

constexpr int kGateMaxExperts = 1024;
constexpr int kGateMaxTopk = 32;             // one lane each

struct GateRule {
  const float* bias;                         // [E], or NULL
  int32_t E, topk;
  int32_t sigmoid, renormalize;
  float scale;
};

namespace {

constexpr uint32_t kFullWarp = 0xFFFFFFFFu;

__device__ __forceinline__ float gate_logit(const void* l, int64_t at, int type) {
  if (type == NVFP4_FP32) return __ldg(static_cast<const float*>(l) + at);
  const unsigned short b = __ldg(static_cast<const unsigned short*>(l) + at);
  return type == NVFP4_BF16 ? bf16_bits_to_f32(b) : __half2float(__ushort_as_half(b));
}

// Larger floats have larger keys, -0 and 0 the same, NaN the largest; 0 is no float's.
__device__ __forceinline__ uint32_t gate_key(float f) {
  if (f != f) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(f + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// The float of a key that is no NaN's.
__device__ __forceinline__ float gate_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ unsigned long long gate_key64(double f) {
  if (f != f) return ~0ull;
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(f + 0.0));
  return b >> 63 ? ~b : b | (1ull << 63);
}

// (a NaN counts as the largest value)
__device__ __forceinline__ float warp_max(float v) {
  return gate_value(__reduce_max_sync(kFullWarp, gate_key(v)));
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullWarp, v, o);
  return v;
}

// Scores of a row of logits; max and total are its softmax's (a row of -infinities
// has no total: all its scores are 0).
struct GateScores {
  float max, inv;
  int sigmoid;
  __device__ __forceinline__ float of(float l) const {
    if (sigmoid) {                                  // (subnormal scores too)
      const float q = expf(-fabsf(l));
      return (l < 0.f ? q : 1.f) / (1.f + q);
    }
    return max == -INFINITY && l == max ? 0.f : expf(l - max) * inv;
  }
};
// A chosen score times a factor that all chosen ones of the row share, by its logit and the
// largest of theirs.  Renormalised weights are ratios of scores: they hold where those leave
// FP32's range (sigmoids of logits below -87; softmax scores that a bias chose, far below the
// row's largest), and only a row whose chosen logits are all -infinities has none.
__device__ __forceinline__ float gate_share(float l, float top, int sigmoid) {
  if (l == -INFINITY) return 0.f;
  if (!sigmoid) return expf(l - top);
  if (l > 0.f) return 1.f / (1.f + expf(-l));
  return expf(l - fminf(top, 0.f)) / (1.f + expf(l));
}
// Scores below this are rounded to fewer bits, or to 0.
constexpr float kGateLeastScore = 2.3509887e-38f;   // 2^-125
template <int L>
__device__ __forceinline__ GateScores gate_scores(const float (&l)[L], int E, int sigmoid) {
  GateScores g{-INFINITY, 1.f, sigmoid};
  if (sigmoid) return g;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < L; ++i) g.max = fmaxf(g.max, l[i]);     // -inf past E
  g.max = warp_max(g.max);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < L; ++i)
    if (lane + 32 * i < E) sum += g.of(l[i]);
  sum = warp_sum(sum);
  g.inv = sum == 0.f ? 0.f : 1.f / sum;
  return g;
}

// The choice on 64-bit keys (with a bias): lane j < topk gets the j-th expert.  (All by
// value: a reference would put the caller's logits into memory for every token.)
template <int L>
struct LaneLogits {
  float v[L];
};
template <int L>
__device__ __noinline__ int gate_choose64(GateRule r, LaneLogits<L> logits, float max) {
  const float (&l)[L] = logits.v;
  const int lane = threadIdx.x & 31;
  unsigned long long key[L];
  double inv = 1.0;
  if (!r.sigmoid) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (lane + 32 * i < r.E && max != -INFINITY)
        sum += exp(static_cast<double>(l[i]) - static_cast<double>(max));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullWarp, sum, o);
    inv = sum == 0.0 ? 0.0 : 1.0 / sum;
  }
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0;
    if (e < r.E) {
      const double x = static_cast<double>(l[i]);
      double s;
      if (r.sigmoid) s = 1.0 / (1.0 + exp(-x));
      else s = max == -INFINITY && l[i] == max ? 0.0 : exp(x - static_cast<double>(max)) * inv;
      key[i] = gate_key64(s + static_cast<double>(__ldg(r.bias + e)));
    }
  }
  int mine = 0;
#pragma unroll 1
  for (int j = 0; j < r.topk; ++j) {
    unsigned long long best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (key[i] > best) { best = key[i]; at = i; }
    const uint32_t hi = static_cast<uint32_t>(best >> 32), lo = static_cast<uint32_t>(best);
    const uint32_t top = __reduce_max_sync(kFullWarp, hi);
    const uint32_t low = __reduce_max_sync(kFullWarp, hi == top ? lo : 0u);
    const int e = static_cast<int>(__reduce_min_sync(
        kFullWarp, hi == top && lo == low ? static_cast<uint32_t>(lane + 32 * at) : ~0u));
    if (j == lane) mine = e;
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (lane + 32 * i == e) key[i] = 0;
  }
  return mine;
}

// The order of n <= 32 experts by sigmoid + bias in 64 bits: lane j has expert e, its logit
// and its score.  One 64-bit exponential a lane; gate_choose64 takes them for all experts.
__device__ __noinline__ int2 gate_reorder64(const float* bias, int n, float logit, int e,
                                            float score) {
  const int lane = threadIdx.x & 31;
  const unsigned long long key =
      lane < n ? gate_key64(1.0 / (1.0 + exp(-static_cast<double>(logit))) +
                            static_cast<double>(__ldg(bias + e)))
               : 0ull;
  int rank = lane < n ? 0 : 32;
  for (int i = 0; i < n; ++i) {
    const unsigned long long k = __shfl_sync(kFullWarp, key, i);
    const int other = __shfl_sync(kFullWarp, e, i);
    if (lane < n && (k > key || (k == key && other < e))) ++rank;
  }
  int2 mine = make_int2(e, __float_as_int(score));
  for (int i = 0; i < n; ++i) {
    const int r = __shfl_sync(kFullWarp, rank, i), x = __shfl_sync(kFullWarp, e, i);
    const float v = __shfl_sync(kFullWarp, score, i);
    if (r == lane) mine = make_int2(x, __float_as_int(v));
  }
  return mine;
}

// l[i]: logit of expert lane + 32 i, -infinity past E.  Lane j < topk gets the j-th
// expert and its weight.
template <int L>
__device__ __forceinline__ void gate_choose(const GateRule& r, const float (&l)[L], int* id,
                                            float* weight) {
  const int lane = threadIdx.x & 31;
  // renormalised softmax weights need no total, nor does the choice without a bias (the largest
  // of the row is then the largest of the chosen)
  const bool total = r.sigmoid || r.bias || !r.renormalize;
  GateScores g{0.f, 1.f, r.sigmoid};
  if (total) {
    g = gate_scores<L>(l, r.E, r.sigmoid);
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < L; ++i) m = fmaxf(m, l[i]);
    g.max = warp_max(m);
  }
  float s[L];
  uint32_t key[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int e = lane + 32 * i;
    s[i] = r.bias && e < r.E ? g.of(l[i]) : l[i];
    key[i] = e < r.E ? gate_key(r.bias ? s[i] + __ldg(r.bias + e) : s[i]) : 0u;
  }
  // Up to four per lane: its experts in order, so that its best is always its first (one token
  // of 128 experts 0.6 us less); sorting eight takes longer than scanning them at every pick
  // (8192 tokens of 256 experts then 1.5 times the time).
  int at[L];
  constexpr bool kSorted = L <= 4;
#pragma unroll
  for (int i = 0; i < L; ++i) at[i] = i;
  float val[L];
#pragma unroll
  for (int i = 0; i < L; ++i) val[i] = s[i];
  if constexpr (kSorted) {
#pragma unroll
    for (int n = L; n > 1; --n)
#pragma unroll
      for (int i = 0; i + 1 < n; ++i) {
        // (equals stay in order: the lower number first)
        const bool swap = key[i] < key[i + 1];
        const uint32_t k0 = key[i];
        const float v0 = val[i];
        const int a0 = at[i];
        key[i] = swap ? key[i + 1] : k0;
        val[i] = swap ? val[i + 1] : v0;
        at[i] = swap ? at[i + 1] : a0;
        key[i + 1] = swap ? k0 : key[i + 1];
        val[i + 1] = swap ? v0 : val[i + 1];
        at[i + 1] = swap ? a0 : at[i + 1];
      }
  }
  // With a bias one more than wanted, and on until a pick is clear of the one before.
  const int picks = r.bias && r.topk < r.E ? r.topk + 1 : r.topk;
  int mine = 0, count = 0;
  float chosen = 0.f, last_s = 0.f, last = 0.f;                   // last: the pick before
  bool near = false, touching = false;
#pragma unroll 1
  for (; count < picks || (touching && r.sigmoid && count < min(r.E, 32)); ++count) {
    uint32_t best = key[0];
    int place = at[0];
    float v = val[0];
    if constexpr (!kSorted) {
#pragma unroll
      for (int i = 1; i < L; ++i)
        if (key[i] > best) { best = key[i]; place = i; v = val[i]; }
    }
    const uint32_t top = __reduce_max_sync(kFullWarp, best);
    const uint32_t who = __ballot_sync(kFullWarp, best == top);
    int from = __ffs(who) - 1;
    if (who & (who - 1))                            // equals: the lowest number
      from = static_cast<int>(__reduce_min_sync(
                 kFullWarp, best == top ? static_cast<uint32_t>(lane + 32 * place) : ~0u)) & 31;
    const int e = __shfl_sync(kFullWarp, lane + 32 * place, from);
    v = __shfl_sync(kFullWarp, v, from);
    if (lane == from) {
#pragma unroll
      for (int i = 0; i < L; ++i) {
        if constexpr (kSorted) {
          key[i] = i + 1 < L ? key[i + 1 < L ? i + 1 : 0] : 0u;
          val[i] = val[i + 1 < L ? i + 1 : 0];
          at[i] = at[i + 1 < L ? i + 1 : 0];
        } else if (i == place) {
          key[i] = 0;
        }
      }
    }
    if (r.bias) {
      const float k = top == 0xFFFFFFFFu ? NAN : gate_value(top);
      // What 32 bits can be off by, with room: a sigmoid two steps of a value (its exponential,
      // sum and quotient are rounded once each), a softmax score 2e-6 of it (its argument and
      // total too), the sum with the bias half a step.
      touching = count > 0 && !(last - k > (r.sigmoid ? 4e-7f : 2e-6f) * (fabsf(last_s) + fabsf(v)) +
                                               1.2e-7f * (fabsf(last) + fabsf(k)));
      near |= touching;
      last_s = v;
      last = k;
    }
    if (count == lane) { mine = e; chosen = v; }
  }
  if (near) {                                       // the same in every lane
    // (all picks are in lanes, and the last one is clear of what follows, or all are picked)
    const bool few = r.sigmoid && count <= 32 && (!touching || count == r.E);
    if (!few) {
      LaneLogits<L> row;
#pragma unroll
      for (int i = 0; i < L; ++i) row.v[i] = l[i];
      mine = gate_choose64<L>(r, row, g.max);
    }
    float logit = 0.f;
    const int n = few ? count : r.topk;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {                   // of the expert's lane
      const int e = __shfl_sync(kFullWarp, mine, j);
      float x = 0.f, v = 0.f;
#pragma unroll
      for (int i = 0; i < L; ++i)
        if (lane + 32 * i == e) { x = l[i]; v = s[i]; }
      x = __shfl_sync(kFullWarp, x, e & 31);
      v = __shfl_sync(kFullWarp, v, e & 31);
      if (j == lane) { logit = x; chosen = v; }
    }
    if (few) {
      const int2 m = gate_reorder64(r.bias, n, logit, mine, chosen);
      mine = m.x;
      chosen = __int_as_float(m.y);
    }
  }
  const bool on = lane < r.topk;
  float w = 0.f;
  // renormalised: by the logits, which are at hand without a bias; with one the scores are, and
  // logits are looked up where a score is too small
  bool shares = r.renormalize && !r.bias;
  float logit = chosen;
  if (r.renormalize && r.bias && __any_sync(kFullWarp, on && chosen < kGateLeastScore)) {
    shares = true;
#pragma unroll 1
    for (int j = 0; j < r.topk; ++j) {              // of the expert's lane
      const int e = __shfl_sync(kFullWarp, mine, j);
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < L; ++i)
        if (lane + 32 * i == e) x = l[i];
      x = __shfl_sync(kFullWarp, x, e & 31);
      if (j == lane) logit = x;
    }
  }
  if (shares) {
    const float top = total ? warp_max(on ? logit : -INFINITY) : g.max;
    if (on) w = gate_share(logit, top, r.sigmoid);
  } else if (on) {
    w = r.bias ? chosen : g.of(chosen);
  }
  if (r.renormalize) {
    const float sum = warp_sum(w);
    w = sum == 0.f ? 0.f : w / sum;
  }
  *id = mine;
  *weight = w * r.scale;
}

}  // namespace
}  // namespace nvfp4
