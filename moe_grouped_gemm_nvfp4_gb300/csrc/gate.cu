// Top-k gate of an MoE layer and its gradient: a warp per token (gate.cuh).
//
// Gradient: with g the gradient of the weights times scale, p and s the scores, w the weights
// renormalised,
//
//   softmax  dl = p (g - sum_j g_j p_j),      renormalised  dl = w (g - sum_j g_j w_j)
//   sigmoid  dl = g s (1 - s),                renormalised  dl = w (1 - s) (g - sum_j g_j w_j)
//
// Where one score (weight) has more than half of the sum, its own gradient is a small difference
// of large values: g is then taken relative to that expert's, which changes no result (the scores
// add up to 1) and makes its term of the sum 0, so that the rest is left without a difference.
//
// All but the first are zero outside the chosen experts and need no other logits, so only the
// chosen ones are read.
//
// Bound: the gate's latency up to some thousand tokens (a chain of topk reductions over the
// warp), then its instructions; its bytes (the logits once) would take a tenth of the time.
// The gradient: latency, then its instructions (its rows are written once, logits read where
// they are needed; a quarter to a third of the copy rate).
// In a graph, FP32 logits, 8 chosen: one token of 128 experts 2.5 to 2.8 us (with a bias 3.8 to
// 4.1), 8192 tokens of 128 6.7 us (with a bias 8.6 to 9.4, softmax 14 where a token's sums are so
// near that it takes 64-bit keys of all experts), of 256 10 us (15), of 512 21 us (31 to 35, with
// such a token 46; as 1024 are done: 57), 65536 of 128 40 us (52 to 58); the gradient 1.7 to 2.1,
// 3.2 to 4.4 (128 experts), 4.2 to 6.1 (256) and 15 to 23 us.
#include <cuda_fp16.h>

#include "gate.h"
#include "rows.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

template <int L>
__global__ void __launch_bounds__(kThreads) topk_gate_kernel(const GateArgs a, int type) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  float l[L];
  auto load = [&](int of) {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int e = lane + 32 * i;
      l[i] = e < a.rule.E ? gate_logit(a.logits, t * a.ld + e, of) : -INFINITY;
    }
  };
  // (one branch outside, so that the loads are on their way together)
  if (type == NVFP4_FP32) load(NVFP4_FP32);
  else if (type == NVFP4_BF16) load(NVFP4_BF16);
  else load(NVFP4_FP16);
  int id;
  float w;
  gate_choose<L>(a.rule, l, &id, &w);
  if (lane < a.rule.topk) {
    a.ids[t * a.rule.topk + lane] = id;
    a.weights[t * a.rule.topk + lane] = w;
  }
}

template <int DT, int L>
__global__ void __launch_bounds__(kThreads) topk_gate_grad_kernel(const GateArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const GateRule& r = a.rule;
  const bool on = lane < r.topk;
  int e = on ? __ldg(a.chosen + t * r.topk + lane) : -1;
  float g = on ? __ldg(a.dweights + t * r.topk + lane) * r.scale : 0.f;
  if (e >= r.E || (on && e < 0)) {
    raise_status(a.status, NVFP4_ERR_DEVICE_CHECK);
    e = -1;
  }
  const bool ok = e >= 0;
  if (!ok) g = 0.f;
  float p[L], inv = 0.f;                           // scores times their total, of all experts
  const bool whole = !r.sigmoid && !r.renormalize;
  const float chosen = ok ? gate_logit(a.logits, t * a.ld + e, DT) : -INFINITY;
  if (whole) {
    float max = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int c = lane + 32 * i;
      p[i] = c < r.E ? gate_logit(a.logits, t * a.ld + c, DT) : -INFINITY;
      max = fmaxf(max, p[i]);
    }
    max = warp_max(max);
#pragma unroll
    for (int i = 0; i < L; ++i) {
      p[i] = lane + 32 * i < r.E && !(max == -INFINITY && p[i] == max) ? expf(p[i] - max) : 0.f;
      sum += p[i];
    }
    sum = warp_sum(sum);
    inv = sum == 0.f ? 0.f : 1.f / sum;
  }
  // what the chosen experts get (whole: the gradient of their scores), then the place of each
  // in its lane's experts
  float d = 0.f;
  const float q = expf(-fabsf(chosen));            // for sigmoids
  if (whole) {
    d = g;
  } else if (r.renormalize) {
    // (the quotient itself: a weight that is alone is 1, and its gradient 0, not p / p's rounding)
    const float share = gate_share(chosen, warp_max(chosen), r.sigmoid);
    const float sum = warp_sum(share);
    const float w = sum == 0.f ? 0.f : share / sum;
    const uint32_t most = __ballot_sync(kFullWarp, w > 0.5f);
    const float shift = most ? __shfl_sync(kFullWarp, g, __ffs(most) - 1) : 0.f;
    d = w * ((g - shift) - warp_sum(w * (g - shift)));
    if (r.sigmoid) d *= (chosen < 0.f ? 1.f : q) / (1.f + q);
    if (!ok) d = 0.f;
  } else if (ok) {                                 // s (1 - s) without the difference
    d = g * (q / ((1.f + q) * (1.f + q)));
  }
  float add[L];
#pragma unroll
  for (int i = 0; i < L; ++i) add[i] = 0.f;
  for (int j = 0; j < r.topk; ++j) {
    const int ej = __shfl_sync(kFullWarp, e, j);
    const float dj = __shfl_sync(kFullWarp, d, j);
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (lane + 32 * i == ej) add[i] += dj;
  }
  if (whole) {
    float own = 0.f, shift = 0.f, back = 0.f;
    bool top = false;
    if (inv > 0.5f) {                              // the same in every lane
#pragma unroll
      for (int i = 0; i < L; ++i)
        if (p[i] == 1.f) { top = true; own = add[i]; }
      const uint32_t most = __ballot_sync(kFullWarp, top);
      shift = most ? __shfl_sync(kFullWarp, own, __ffs(most) - 1) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < L; ++i) {
      p[i] *= inv;
      add[i] -= shift;
      back = fmaf(p[i], add[i], back);
    }
    back = warp_sum(back);
#pragma unroll
    for (int i = 0; i < L; ++i) add[i] = p[i] * (add[i] - back);
  }
  using Bits = typename Elem<DT>::Bits;
  Bits* out = static_cast<Bits*>(a.dlogits) + t * r.E;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int c = lane + 32 * i;
    if (c < r.E) out[c] = static_cast<Bits>(f32_to_elem<DT>(add[i]));
  }
}

template <int DT>
cudaError_t grad(const GateArgs& a, unsigned g, cudaStream_t s) {
  const int E = a.rule.E;
  if (E <= 64) topk_gate_grad_kernel<DT, 2><<<g, kThreads, 0, s>>>(a);
  else if (E <= 128) topk_gate_grad_kernel<DT, 4><<<g, kThreads, 0, s>>>(a);
  else if (E <= 256) topk_gate_grad_kernel<DT, 8><<<g, kThreads, 0, s>>>(a);
  else if (E <= 512) topk_gate_grad_kernel<DT, 16><<<g, kThreads, 0, s>>>(a);
  else topk_gate_grad_kernel<DT, 32><<<g, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_topk_gate(const GateArgs& a, int dtype, cudaStream_t s) {
  const int64_t blocks = (a.T + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  const unsigned g = static_cast<unsigned>(blocks);
  const int E = a.rule.E;
  if (E <= 64) topk_gate_kernel<2><<<g, kThreads, 0, s>>>(a, dtype);
  else if (E <= 128) topk_gate_kernel<4><<<g, kThreads, 0, s>>>(a, dtype);
  else if (E <= 256) topk_gate_kernel<8><<<g, kThreads, 0, s>>>(a, dtype);
  else if (E <= 512) topk_gate_kernel<16><<<g, kThreads, 0, s>>>(a, dtype);
  else topk_gate_kernel<32><<<g, kThreads, 0, s>>>(a, dtype);
  return cudaGetLastError();
}

cudaError_t launch_topk_gate_grad(const GateArgs& a, int dtype, cudaStream_t s) {
  const int64_t blocks = (a.T + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  const unsigned g = static_cast<unsigned>(blocks);
  if (dtype == NVFP4_BF16) return grad<NVFP4_BF16>(a, g, s);
  if (dtype == NVFP4_FP16) return grad<NVFP4_FP16>(a, g, s);
  return grad<NVFP4_FP32>(a, g, s);
}

}  // namespace nvfp4
