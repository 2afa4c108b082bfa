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
// can swap experts.  Each sum has a bound of its error (gate_error), which grows with the score
// and not with the sum.  Where the bounds of two picks that follow each other touch, or that of
// any expert left out reaches the lowest of the picks', these experts (or, where they are too
// many, all) are ordered again on 64-bit keys.  64-bit exponentials for all would take longer
// than everything else here.
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
    // (times inv there too: it is NaN where a NaN stands among infinities)
    return (max == -INFINITY && l == max ? 0.f : expf(l - max)) * inv;
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
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    double v = 0.0;                                 // sigmoid, or softmax before its total
    if (lane + 32 * i < r.E) {
      const double x = static_cast<double>(l[i]);
      if (r.sigmoid) v = 1.0 / (1.0 + exp(-x));
      else if (!(max == -INFINITY && l[i] == max)) v = exp(x - static_cast<double>(max));
    }
    sum += v;
    key[i] = static_cast<unsigned long long>(__double_as_longlong(v));
  }
  double inv = 1.0;
  if (!r.sigmoid) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullWarp, sum, o);
    inv = sum == 0.0 ? 0.0 : 1.0 / sum;
  }
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int e = lane + 32 * i;
    // (rounded by itself: equal scores stay equal whichever products the compiler would fuse)
    const double s = __dmul_rn(__longlong_as_double(static_cast<long long>(key[i])), inv);
    key[i] = e < r.E ? gate_key64(__dadd_rn(s, static_cast<double>(__ldg(r.bias + e)))) : 0ull;
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

// What the 32-bit sum k = s + bias can be off by, with room.  A sigmoid: its exponential (two
// steps, of an exact argument), its sum and quotient, 6 * 2^-24 of it.  A softmax score, in units
// of 2^-24 of it: |l - max| by its argument's rounding, which is -log(score) at most; 4 by the
// exponential; its total's terms likewise (4 and less than 7, the mean of |l - max|), L + 4
// additions, quotient and product.  The sum itself half a step (a whole one is taken: the
// bounds' own sums round too).  Subnormal scores and sums: some of the smallest steps.
// MOST: with the smallest score's logarithm, -105, for any.
template <int L, bool MOST>
__device__ __forceinline__ float gate_error(float s, float k, int sigmoid) {
  float of_score = 4e-7f;
  if (!sigmoid)
    of_score = 6.2e-8f * (L + 28.f + (MOST ? 105.f : -__logf(fminf(fmaxf(s, 1.2e-38f), 1.f))));
  return of_score * s + 1.2e-7f * fabsf(k) + 1e-44f;
}
__device__ __forceinline__ bool is_finite(float k) { return fabsf(k) < INFINITY; }

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
  int mine = 0;
  float chosen = 0.f;
#pragma unroll 1
  for (int count = 0; count < r.topk; ++count) {
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
    if (count == lane) { mine = e; chosen = v; }
    // (no instruction, but the compiler's order of the loop is 12% faster around it, with a bias
    // or without: 65536 tokens of 128 experts 44.5 -> 39.6 us)
    if (r.bias) asm volatile("" ::: "memory");
  }
  const bool on = lane < r.topk;
  // Lanes: the picks.  An infinity or a NaN is certain, and so is its place.
  bool near = false;
  uint32_t may = 0;                                 // experts left that may belong before a pick
  int more = 0;
  if (r.bias) {
    const float k = chosen + __ldg(r.bias + mine);
    const float error = gate_error<L, false>(chosen, k, r.sigmoid);
    const bool sure = !on || !is_finite(k);
    const float least = sure ? INFINITY : k - error;
    const float before = __shfl_up_sync(kFullWarp, least, 1);
    const float low = gate_value(__reduce_min_sync(kFullWarp, gate_key(least)));
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const float x = gate_value(key[i]);
      if (key[i] != 0 && is_finite(x) && !(x + gate_error<L, true>(val[i], x, r.sigmoid) < low))
        may |= 1u << i;
    }
    if (!r.sigmoid && __any_sync(kFullWarp, may != 0)) {
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const float x = gate_value(key[i]);
        if (x + gate_error<L, false>(val[i], x, 0) < low) may &= ~(1u << i);
      }
    }
    more = __reduce_add_sync(kFullWarp, __popc(may));
    near = more > 0 || __any_sync(kFullWarp, lane > 0 && !sure && !(k + error < before));
  }
  if (near) {                                       // the same in every lane
    const bool few = r.sigmoid && r.topk + more <= 32;
    if (!few) {
      LaneLogits<L> row;
#pragma unroll
      for (int i = 0; i < L; ++i) row.v[i] = l[i];
      mine = gate_choose64<L>(r, row, g.max);
      more = 0;
    }
#pragma unroll 1
    for (int j = r.topk; j < r.topk + more; ++j) {  // those behind the picks, one a lane
      const int from = __ffs(__ballot_sync(kFullWarp, may != 0)) - 1;
      const int i0 = __ffs(may) - 1;
      int e = 0;
#pragma unroll
      for (int i = 0; i < L; ++i)
        if (i == i0) e = lane + 32 * at[i];
      e = __shfl_sync(kFullWarp, e, from);
      if (lane == from) may &= may - 1;
      if (j == lane) mine = e;
    }
    float logit = 0.f;
    const int n = r.topk + more;
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
