// Routing: from each token's logits to its topk experts and their weights.
//
// Mathematics, for a row of logits l:
//   s = 1 / (1 + exp(-l)) or exp(l - max) / sum exp(l - max)
//   v = s + bias; without a bias the order of v is that of l, and l stands in
//       for it (but where groups count by sums of two)
//   groups: value = the sum of the best group_best v; the best topk_groups
//       groups stay, equal ones by their number
//   picks: the topk largest v of those, in descending order, equal ones by
//       their number
//   w = s, or s / (sum of the picks' s), times scale.
// A logit that is NaN or -infinity leaves its expert out (of the softmax's
// sum too), so does a bias that is; +infinity counts as the largest fp32. All
// of it in 64 bits: which of two near scores is larger decides whole numbers,
// and fp32 scores of one row come within each other's rounding about once in
// a few hundred rows. Renormalised weights are quotients of scores whose
// largest may underflow; a common factor exp(-min(largest logit, 0)) is taken
// out first, so they are the quotients' values all the same.
#include <hip/hip_runtime.h>
#include <float.h>
#include <stdint.h>

#include "pick.h"

namespace llmoe {
namespace {

constexpr int kRowsAtOnce = 4;  // wavefronts of a workgroup, a row each

__device__ __forceinline__ double none() { return -__builtin_inf(); }

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmax(v, __shfl_xor(v, d, 64));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// A logit or bias as it counts: NaN as -infinity, at most the largest fp32.
__device__ __forceinline__ float counted(float x) { return x == x ? fminf(x, FLT_MAX) : -__builtin_inff(); }

__device__ __forceinline__ float logit_at(const PickParams& P, int64_t at) {
  if (P.bf16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(P.logits)[at] << 16);
  return static_cast<const float*>(P.logits)[at];
}

__device__ __forceinline__ double sigmoid(double l) { return 1.0 / (1.0 + exp(-l)); }

// Weights of the picks of one row and their stores: lane k < topk holds pick
// k, its expert (-1: none) and its logit; m and z are the softmax's.
__device__ __forceinline__ void put_picks(const PickParams& P, int64_t row, int lane, int e, float logit, double m,
                                          double z) {
  const bool on = lane < P.topk && e >= 0;
  const double l = logit;
  double w = 0.0;
  if (P.renormalize) {
    const double top = wave_max(on ? l : none());
    if (P.sigmoid) {
      const double shift = fmin(top, 0.0);
      w = l >= 0.0 ? 1.0 / (1.0 + exp(-l)) : exp(l - shift) / (1.0 + exp(l));
    } else {
      w = exp(l - top);
    }
    w = on ? w : 0.0;
    const double sum = wave_sum(w);
    w = on ? w / sum : 0.0;
  } else if (on) {
    w = P.sigmoid ? sigmoid(l) : exp(l - m) / z;
  }
  if (lane < P.topk) {
    P.topk_idx[row * P.topk + lane] = e;
    P.topk_weights[row * P.topk + lane] = (float)(w * (double)P.scale);
  }
}

// V: experts a lane holds, expert lane + 64 i in place i.
template <int V>
__global__ void __launch_bounds__(kRowsAtOnce * 64) pick_kernel(const PickParams P) {
  extern __shared__ double values_raw[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = P.num_experts, per = E / P.num_groups;
  double* values = values_raw + wave * E;
  const int valid = P.num_valid ? *P.num_valid : P.num_tokens;
  for (int64_t row = (int64_t)blockIdx.x * kRowsAtOnce + wave; row < P.num_tokens;
       row += (int64_t)gridDim.x * kRowsAtOnce) {
    if (row >= valid) {
      put_picks(P, row, lane, -1, 0.0f, 0.0, 1.0);
      continue;
    }
    float l[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      l[i] = e < E ? counted(logit_at(P, row * E + e)) : -__builtin_inff();
    }
    double m = 0.0, z = 1.0;
    if (!P.sigmoid) {
      m = none();
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmax(m, (double)l[i]);
      m = wave_max(m);
      z = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) z += l[i] > -__builtin_inff() ? exp((double)l[i] - m) : 0.0;
      z = wave_sum(z);
    }
    auto score = [&](float x) { return P.sigmoid ? sigmoid(x) : exp((double)x - m) / z; };

    double v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      const bool in = l[i] > -__builtin_inff();
      if (P.bias) {
        const float b = e < E ? counted(P.bias[e]) : -__builtin_inff();
        v[i] = in && b > -__builtin_inff() ? score(l[i]) + (double)b : none();
      } else {
        v[i] = l[i];
      }
    }
    if (P.num_groups > 1) {
      const bool sums = !P.bias && P.group_best == 2;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        if (e < E) values[e] = sums && l[i] > -__builtin_inff() ? score(l[i]) : v[i];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      double best = none(), second = none();
      if (lane < P.num_groups) {
        for (int j = 0; j < per; ++j) {
          const double x = values[lane * per + j];
          second = fmax(second, fmin(best, x));
          best = fmax(best, x);
        }
      }
      const double mine = P.group_best == 2 ? best + second : best;
      int before = 0;
      for (int g = 0; g < P.num_groups; ++g) {
        const double other = __shfl(mine, g, 64);
        before += other > mine || (other == mine && g < lane);
      }
      const uint64_t kept = __ballot(lane < P.num_groups && before < P.topk_groups);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        if (e < E && !(kept >> (e / per) & 1)) v[i] = none();
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }

    int pick = -1;
    float pick_l = 0.0f;
    for (int k = 0; k < P.topk; ++k) {
      double best = none();
      int e = INT32_MAX;
      float bl = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (v[i] > best) best = v[i], e = lane + 64 * i, bl = l[i];
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double ov = __shfl_xor(best, d, 64);
        const int oe = __shfl_xor(e, d, 64);
        const float ol = __shfl_xor(bl, d, 64);
        if (ov > best || (ov == best && oe < e)) best = ov, e = oe, bl = ol;
      }
      if (!(best > none())) break;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 64 * i == e) v[i] = none();
      if (lane == k) pick = e, pick_l = bl;
    }
    put_picks(P, row, lane, pick, pick_l, m, z);
  }
}

template <int V>
hipError_t launch(const PickParams& p, hipStream_t stream) {
  const int64_t needed = ((int64_t)p.num_tokens + kRowsAtOnce - 1) / kRowsAtOnce;
  const unsigned blocks = (unsigned)(needed < 1 << 16 ? needed : 1 << 16);
  const uint32_t lds = p.num_groups > 1 ? kRowsAtOnce * p.num_experts * 8u : 0u;
  pick_kernel<V><<<blocks, kRowsAtOnce * 64, lds, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_pick(const PickParams& p, hipStream_t stream) {
  if (p.num_tokens == 0) return hipSuccess;
  if (p.num_experts <= 64) return launch<1>(p, stream);
  if (p.num_experts <= 128) return launch<2>(p, stream);
  if (p.num_experts <= 256) return launch<4>(p, stream);
  if (p.num_experts <= 512) return launch<8>(p, stream);
  if (p.num_experts <= 1024) return launch<16>(p, stream);
  return launch<64>(p, stream);
}

}  // namespace llmoe
