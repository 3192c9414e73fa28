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
// sum too), so does a bias that is; +infinity counts as the largest fp32.
// Which of two near scores is larger decides whole numbers, and fp32 scores of
// one row come within each other's rounding about once in a few hundred rows:
// the order is that of 64 bits. Renormalised weights are quotients of scores whose
// largest may underflow; a common factor exp(-min(largest logit, 0)) is taken
// out first, so they are the quotients' values all the same.
//
// Design: four rows a wavefront, 16 lanes each (pick_rows_kernel), whose values
// are in registers, the lanes read each other by row rotations, and the few
// values that can be among the picks meet in LDS to be ranked. fp32 values
// decide wherever they are further apart than they may be off; those that are
// not are taken again to 1e-10, and a row that this does not settle is done by a
// whole wavefront in 64 bits (exact_row), as is every row of the other counts of
// experts and groups. Not settled are sums of groups that are equal numbers, and,
// of scores with a bias, more than 16 that reach a bound for the topk-th: many
// equal ones, or all of the few lanes that are left where few groups stay (16384
// tokens of 256 experts in 8 groups, 8 picks: 2 groups stay 54 us, 1 stays 100).
//
// Bound: 16384 tokens of 256 experts (fp32, sigmoid with a bias, 8 groups, 4
// stay, 8 picks; 18 MB) take 11.6 us a launch, 1.5 TB/s: 1100 vector instructions a wavefront,
// many in 64 bits, for four wavefronts a SIMD, each a chain of row rotations
// behind one another. One token takes 4.5 us, a launch and one such chain.
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

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v, uint32_t old = 0) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v), __float_as_uint(v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32 | dpp<CTRL>((uint32_t)u)));
}
constexpr int kRor = 0x120, kShl = 0x100, kShr = 0x110;  // by n lanes of a row of 16

__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp<kRor + 8>(v));
  v = fmaxf(v, dpp<kRor + 4>(v));
  v = fmaxf(v, dpp<kRor + 2>(v));
  return fmaxf(v, dpp<kRor + 1>(v));
}
__device__ __forceinline__ double row_sum(double v) {
  v += dpp<kRor + 8>(v);
  v += dpp<kRor + 4>(v);
  v += dpp<kRor + 2>(v);
  return v + dpp<kRor + 1>(v);
}

__device__ __forceinline__ uint64_t row_max(uint64_t v) {
  auto with = [&](uint32_t hi, uint32_t lo) {
    const uint64_t other = (uint64_t)hi << 32 | lo;
    v = other > v ? other : v;
  };
  with(dpp<kRor + 8>((uint32_t)(v >> 32)), dpp<kRor + 8>((uint32_t)v));
  with(dpp<kRor + 4>((uint32_t)(v >> 32)), dpp<kRor + 4>((uint32_t)v));
  with(dpp<kRor + 2>((uint32_t)(v >> 32)), dpp<kRor + 2>((uint32_t)v));
  with(dpp<kRor + 1>((uint32_t)(v >> 32)), dpp<kRor + 1>((uint32_t)v));
  return v;
}

// How many of a row's 16 values are larger.
template <int N = 1>
__device__ __forceinline__ uint32_t rank(uint64_t v) {
  const uint64_t other = (uint64_t)dpp<kRor + N>((uint32_t)(v >> 32)) << 32 | dpp<kRor + N>((uint32_t)v);
  if constexpr (N < 15) return (other > v) + rank<N + 1>(v);
  else return other > v;
}

// The same of values and, where those are equal, smaller numbers.
template <int N = 1>
__device__ __forceinline__ uint32_t rank_by(double v, uint32_t number) {
  const double ov = dpp<kRor + N>(v);
  const uint32_t on = dpp<kRor + N>(number);  // lanes read each other: never behind a condition
  const uint32_t before = ov > v || (ov == v && on < number);
  if constexpr (N < 15) return before + rank_by<N + 1>(v, number);
  else return before;
}
__device__ __forceinline__ double row_max(double v) {
  v = fmax(v, dpp<kRor + 8>(v));
  v = fmax(v, dpp<kRor + 4>(v));
  v = fmax(v, dpp<kRor + 2>(v));
  return fmax(v, dpp<kRor + 1>(v));
}

// exp(x) for x <= 0, 1e-11 off at most: 2^n times the series of the rest,
// |r| <= ln(2) / 2, whose tenth power over 10! is 7e-12.
__device__ __forceinline__ double exp_series(double x) {
  x = fmax(x, -750.0);
  const double n = rint(x * 1.4426950408889634);
  const double r = __builtin_fma(n, -0.69314718055994531, x);
  double v = 1.0 / 362880;
  v = __builtin_fma(v, r, 1.0 / 40320);
  v = __builtin_fma(v, r, 1.0 / 5040);
  v = __builtin_fma(v, r, 1.0 / 720);
  v = __builtin_fma(v, r, 1.0 / 120);
  v = __builtin_fma(v, r, 1.0 / 24);
  v = __builtin_fma(v, r, 1.0 / 6);
  v = __builtin_fma(v, r, 0.5);
  v = __builtin_fma(v, r, 1.0);
  v = __builtin_fma(v, r, 1.0);
  return __builtin_ldexp(v, (int)n);
}

__device__ __forceinline__ double sigmoid_series(double x) {
  const double t = exp_series(-fabs(x)), one = 1.0 / (1.0 + t);
  return x >= 0.0 ? one : t * one;
}

// Weights of a row's picks and their stores. Lane k < topk of a row of 16 holds
// pick k, its expert (-1: none) and its logit; m and z are the softmax's. What
// is rounded to fp32 is 1e-10 off at most.
__device__ __forceinline__ void put(const PickParams& P, int64_t row, int k, int e, float logit, double m, double z,
                                    bool store) {
  const bool on = k < P.topk && e >= 0;
  const double l = on ? (double)logit : 0.0;
  double w;
  if (P.sigmoid) {
    const double x = exp_series(-fabs(l)), one = 1.0 / (1.0 + x);
    w = l >= 0.0 ? one : x * one;
    if (P.renormalize) {
      // all below zero: without the common factor, that may be all there is
      const float top = row_max(on ? logit : -__builtin_inff());
      if (__ballot(top < 0.0f)) w = top < 0.0f ? exp_series(on ? l - (double)top : 0.0) * one : w;
    }
  } else if (P.renormalize) {
    const float top = row_max(on ? logit : -__builtin_inff());
    w = exp_series(on ? l - (double)top : 0.0);
  } else {
    w = exp_series(on ? l - m : 0.0) / z;
  }
  w = on ? w : 0.0;
  if (P.renormalize) {
    const double sum = row_sum(w);  // of all lanes, so outside the choice
    w = on ? w / sum : 0.0;
  }
  if (store && k < P.topk) {
    P.topk_idx[row * P.topk + k] = e;
    P.topk_weights[row * P.topk + k] = (float)(w * (double)P.scale);
  }
}

// A row by a whole wavefront, everything in 64 bits. V: experts a lane holds,
// expert lane + 64 i in place i; values: LDS for the experts' values, if there
// are groups.
template <int V>
__device__ __forceinline__ void exact_row(const PickParams& P, int64_t row, int lane, double* values) {
  const int E = P.num_experts, per = E / P.num_groups;
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
  put(P, row, lane, pick, pick_l, m, z, lane < 16);
}

template <int V>
__global__ void __launch_bounds__(kRowsAtOnce * 64) pick_kernel(const PickParams P) {
  extern __shared__ double values_raw[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int valid = P.num_valid ? *P.num_valid : P.num_tokens;
  for (int64_t row = (int64_t)blockIdx.x * kRowsAtOnce + wave; row < P.num_tokens;
       row += (int64_t)gridDim.x * kRowsAtOnce) {
    if (row >= valid) put(P, row, lane, -1, 0.0f, 0.0, 1.0, lane < 16);
    else exact_row<V>(P, row, lane, values_raw + wave * P.num_experts);
  }
}

// Four rows a wavefront, 16 lanes each: the choice by fp32 values wherever
// those decide it, and by exact_row where two that matter are within what
// fp32 may be off by.

// Values' bits in an order that unsigned numbers have.
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return u ^ ((uint64_t)((int64_t)u >> 63) | 1ull << 63);
}

// exact_row as a call of its own: rare, and its code and registers are not the
// kernel's. It takes the parameters where the kernel's arguments stand (copies
// of them for the call would be read from memory by the kernel, too).
template <int V>
__device__ __noinline__ void exact_row_apart(const PickParams* P, int64_t row, int lane, double* values) {
  const PickParams p = *P;
  exact_row<V>(p, row, lane, values);
}
__device__ __forceinline__ const PickParams* kernel_params() {
  return (const PickParams*)__builtin_amdgcn_kernarg_segment_ptr();
}

__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((uint32_t)((int32_t)~u >> 31) | 0x80000000u));
}

typedef uint32_t Words4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t Words2 __attribute__((ext_vector_type(2), aligned(4)));
// N words from a 4-byte aligned address.
template <int N>
__device__ __forceinline__ void load_words(const void* from, uint32_t (&w)[N]) {
  const uint32_t* at = static_cast<const uint32_t*>(from);
  if constexpr (N == 2) {
    const Words2 v = *reinterpret_cast<const Words2*>(at);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const Words4 v = *reinterpret_cast<const Words4*>(at + i);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  }
}

// What the rows kernel goes by: values that are the logits, whose order is
// exact, or scores with a bias.
enum : int { kByLogits = 0, kBySigmoid = 1, kBySoftmax = 2 };

// A row of 16 lanes holds a row's values, V a lane: expert lane * own + i if
// the lanes have runs of experts (VEC: of V, read 16 bytes at a time), else
// 16 i + lane.
template <int V, bool VEC, int KIND>
__global__ void __launch_bounds__(kRowsAtOnce * 64) pick_rows_kernel(const PickParams P) {
  extern __shared__ double values_raw[];
  constexpr bool SCORED = KIND != kByLogits;
  __shared__ uint64_t found[kRowsAtOnce][4][17];
  __shared__ float found_l[kRowsAtOnce][4][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, sub = lane >> 4;
  const int E = P.num_experts;
  const bool runs = VEC || P.num_groups > 1;
  const int own = VEC ? V : (E + 15) / 16;
  const float none32 = -__builtin_inff();
  const bool sums = P.num_groups > 1 && P.group_best == 2;
  auto expert = [&](int i) { return runs ? l16 * own + i : 16 * i + l16; };
  for (int64_t row0 = ((int64_t)blockIdx.x * kRowsAtOnce + wave) * 4; row0 < P.num_tokens;
       row0 += (int64_t)gridDim.x * kRowsAtOnce * 4) {
    // every load goes out before any is used; rows behind the last read it again
    const int64_t row = row0 + sub, from = row < P.num_tokens ? row : P.num_tokens - 1;
    const int valid = P.num_valid ? *P.num_valid : P.num_tokens;
    float l[V], b[V];
    if constexpr (VEC) {
      uint32_t w[V], u[V];
      if (P.bf16) {
        uint32_t h[V / 2];
        load_words(static_cast<const uint8_t*>(P.logits) + (from * 16 + l16) * (V * 2), h);
        if (SCORED) load_words(P.bias + l16 * V, u);
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = i & 1 ? h[i / 2] & 0xFFFF0000u : h[i / 2] << 16;
      } else {
        load_words(static_cast<const uint8_t*>(P.logits) + (from * 16 + l16) * (V * 4), w);
        if (SCORED) load_words(P.bias + l16 * V, u);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        l[i] = __uint_as_float(w[i]);
        if (SCORED) b[i] = __uint_as_float(u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = expert(i);
        const bool in = e < E && (!runs || i < own);
        l[i] = in ? logit_at(P, from * E + e) : none32;
        if (SCORED) b[i] = in ? P.bias[e] : none32;
      }
    }
    const bool live = row < P.num_tokens && row < valid;
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = counted(l[i]);

    // The softmax's sum, in 64 bits, where anything needs it. The scores of
    // groups without a bias need no sum: it is the same for all.
    double m = 0.0, z = 1.0;
    float key[V];
    if (KIND == kBySoftmax || (KIND == kByLogits && !P.sigmoid && (sums || !P.renormalize))) {
      float top = none32;
#pragma unroll
      for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
      m = row_max(top);
      z = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const double x = l[i] > none32 ? exp_series((double)l[i] - m) : 0.0;
        if (SCORED) key[i] = (float)x;
        z += x;
        if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // a few at a time, for the registers
      }
      z = row_sum(z);
    }
    // A score to 1e-10 or better; those that a choice hangs on once fp32 cannot
    // tell, and the weights.
    auto score64 = [&](float x) {
      if (KIND == kBySigmoid || (KIND == kByLogits && P.sigmoid)) return sigmoid_series(x);
      return exp_series((double)x - m) / z;
    };
    // the values
    auto sigmoid32 = [](float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); };
    const float inv = (float)(1.0 / z);
    auto score32 = [&](float x) { return P.sigmoid ? sigmoid32(x) : __expf(x - (float)m) * inv; };
    if constexpr (SCORED) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float s = KIND == kBySigmoid ? sigmoid32(l[i]) : key[i] * inv;
        key[i] = l[i] > none32 ? s + counted(b[i]) : none32;
      }
    } else {
      // one kind of zero: equal logits are equal numbers
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = l[i] + 0.0f;
    }

    // the lane's best two
    float first = none32, second = none32;
    auto enter = [&](float x) {
      second = __builtin_amdgcn_fmed3f(first, second, x);
      first = fmaxf(first, x);
    };
#pragma unroll
    for (int i = 0; i < V; ++i) enter(key[i]);

    // groups: 16 / num_groups lanes each
    bool unsure = false;
    if (P.num_groups > 1) {
      const float lane_first = first, lane_second = second;
      if (!SCORED && sums) {
        first = second = none32;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          enter(l[i] > none32 ? score32(l[i]) : none32);
        }
      }
      const int lanes = 16 / P.num_groups;
      auto join = [&](float of, float os) {
        second = fmaxf(fmaxf(second, os), fminf(first, of));
        first = fmaxf(first, of);
      };
      // with the neighbour, the neighbouring pair, the neighbouring four
      if (lanes >= 2) join(dpp<0xB1>(first), dpp<0xB1>(second));
      if (lanes >= 4) join(dpp<0x4E>(first), dpp<0x4E>(second));
      if (lanes >= 8) join(dpp<0x141>(first), dpp<0x141>(second));
      // (a sum below fp32's values is still that of a group that has its two)
      const float mine = !sums ? first : second > none32 ? fmaxf(first + second, -FLT_MAX) : none32;
      // every lane of a better group stands before this one's
      const uint32_t stay = P.topk_groups * lanes;
      bool kept = rank((uint64_t)ordered(mine) << 32 | (uint32_t)(16 - l16 / lanes)) < stay;
      if (SCORED || sums) {
        // the nearest values on both sides of the border, and how large
        // anything in them is
        const float in = -row_max(kept ? -mine : none32), out = row_max(kept ? none32 : mine);
        const float size = row_max(first > none32 ? fabsf(first) + (sums && second > none32 ? fabsf(second) : 0.0f) : 0.0f);
        const float off = 0x1p-19f + 0x1p-20f * size;
        const bool tight = out > none32 && !(in - out > off);
        if (__ballot(tight)) {
          // The values of the groups again, to 1e-10: the best two (or one) of
          // every member within `off` of the second (first), among which they
          // are, however near to each other
          const float from = (sums ? second : first) - off;
          double top1 = none(), top2 = none();
          auto enter64 = [&](double t1, double t2) {
            top2 = fmax(fmax(top2, t2), fmin(top1, t1));
            top1 = fmax(top1, t1);
          };
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float x = !SCORED && sums ? (l[i] > none32 ? score32(l[i]) : none32) : key[i];
            if (x > none32 && x >= from) enter64(score64(l[i]) + (SCORED ? (double)counted(b[i]) : 0.0), none());
          }
          if (lanes >= 2) enter64(dpp<0xB1>(top1), dpp<0xB1>(top2));
          if (lanes >= 4) enter64(dpp<0x4E>(top1), dpp<0x4E>(top2));
          if (lanes >= 8) enter64(dpp<0x141>(top1), dpp<0x141>(top2));
          const double exact = sums ? top1 + top2 : top1;
          const bool kept64 = rank((uint64_t)ordered(exact)) < stay;
          const double in64 = -row_max(kept64 ? -exact : none()), out64 = row_max(kept64 ? none() : exact);
          const double off64 = 0x1p-30 + 0x1p-48 * (double)size;
          // (the border of 64 bits must not be a tie either: equal values stay
          // or go together there, and then not as many groups stay as should)
          const uint32_t staying = (uint32_t)__popcll(__ballot(kept64) >> (lane & 48) & 0xFFFF);
          const bool left = staying != stay || !(in64 - out64 > off64);
          unsure = tight && row_max(left ? 1.0f : 0.0f) > 0.0f;
          kept = tight ? kept64 : kept;
        }
      }
      first = kept ? lane_first : none32;
      second = kept ? lane_second : none32;
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = kept ? key[i] : none32;
    }

    // A bound that at least topk values reach: the topk-th largest of the
    // lanes' best two (none, where the groups that stay have fewer lanes than that).
    float bound = none32;
    for (int k = 0; k < P.topk; ++k) {
      bound = row_max(first);
      const bool taken = first == bound;
      first = taken ? second : first;
      second = taken ? none32 : second;
    }
    // Values nearer than this to each other may be in another order: a score's
    // error is below 5 2^-24, its sum's with the bias half a step.
    auto near = [&](float v) { return SCORED ? 0x1p-20f + 0x1p-21f * fabsf(v) : 0.0f; };
    const float least = bound > none32 ? fmaxf(bound - near(bound), -FLT_MAX) : -FLT_MAX;

    // the values that reach it, side by side in LDS
    uint32_t count = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) count += key[i] >= least;
    uint32_t upto = count;
    upto += dpp<kShr + 1>(upto);
    upto += dpp<kShr + 2>(upto);
    upto += dpp<kShr + 4>(upto);
    upto += dpp<kShr + 8>(upto);
    uint32_t all = upto;
    all = max(all, dpp<kRor + 8>(all));
    all = max(all, dpp<kRor + 4>(all));
    all = max(all, dpp<kRor + 2>(all));
    all = max(all, dpp<kRor + 1>(all));
    uint32_t at = upto - count;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] >= least && at < 16) {
        found[wave][sub][at] = (uint64_t)ordered(key[i]) << 32 | (0xFFFFu - expert(i));
        if (SCORED) found_l[wave][sub][at] = l[i];
        ++at;
      }
    uint64_t many = 0;  // lane k: pick k, where there are more than 16
    if constexpr (SCORED) {
      unsure |= all > 16;
    } else if (__ballot(all > 16)) {
      uint64_t last = ~0ull;
      for (int k = 0; k < P.topk; ++k) {
        uint64_t next = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const uint64_t v = (uint64_t)ordered(key[i]) << 32 | (0xFFFFu - expert(i));
          if (key[i] > none32 && v < last && v > next) next = v;
        }
        last = row_max(next);
        if (l16 == k) many = last;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const bool in = (uint32_t)l16 < all;
    const uint64_t mine = in ? found[wave][sub][l16] : 0;
    const float mine_l = SCORED && in ? found_l[wave][sub][l16] : 0.0f;
    // a value's place is the number of larger ones (of equal ones with a
    // smaller expert)
    const uint32_t place = rank(mine);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (in) {
      found[wave][sub][place] = mine;
      if (SCORED) found_l[wave][sub][place] = mine_l;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    uint64_t pick = in ? found[wave][sub][l16] : 0;
    if (!SCORED && all > 16) pick = many;
    const float pick_key = unordered((uint32_t)(pick >> 32));
    float pick_l = !SCORED ? pick_key : in ? found_l[wave][sub][l16] : 0.0f;
    int e = pick ? (int)(0xFFFFu - (uint32_t)pick) : -1;
    if constexpr (SCORED) {
      // neighbours too near to tell
      const float next = dpp<kShl + 1>(pick_key);
      const bool last = l16 >= P.topk || (uint32_t)l16 + 1 >= all || l16 == 15;
      const bool close = !last && !(pick_key - next > near(fmaxf(fabsf(pick_key), fabsf(next))));
      if (__ballot(close)) {
        // the row's values again, to 1e-10, and their places by those
        const float pick_b = in ? counted(P.bias[e]) : 0.0f;
        const double v = in ? score64(pick_l) + (double)pick_b : none();
        const uint32_t again = rank_by(v, (uint32_t)e);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (in) {
          found[wave][sub][again] = (uint64_t)__float_as_uint(pick_b) << 32 | (uint32_t)e;
          found_l[wave][sub][again] = pick_l;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (in) {
          e = (int)(uint32_t)found[wave][sub][l16];
          pick_l = found_l[wave][sub][l16];
        }
        const float in_b = in ? __uint_as_float((uint32_t)(found[wave][sub][l16] >> 32)) : 0.0f;
        const double in_v = in ? score64(pick_l) + (double)in_b : none();
        const double next_v = dpp<kShl + 1>(in_v);
        const float next_l = dpp<kShl + 1>(pick_l), next_b = dpp<kShl + 1>(in_b);
        const bool same = pick_l == next_l && in_b == next_b;
        unsure |= !last && !same && !(in_v - next_v > 0x1p-30 + 0x1p-48 * fabs(in_v));
      }
    }
    // unsure rows again by the whole wavefront; the others' weights
    const uint64_t again = __ballot(unsure && live);
    put(P, row, l16, live ? e : -1, pick_l, m, z, row < P.num_tokens && !(again >> (lane & 48) & 0xFFFF));
    __builtin_amdgcn_wave_barrier();  // found is read before the next rows' values are written
    for (int r = 0; r < 4; ++r)
      if (again >> (16 * r) & 0xFFFF) exact_row_apart<(V + 3) / 4>(kernel_params(), row0 + r, lane, values_raw + wave * E);
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

template <int V, bool VEC>
hipError_t launch_rows(const PickParams& p, hipStream_t stream) {
  constexpr int ROWS = 4 * kRowsAtOnce;
  const int64_t needed = ((int64_t)p.num_tokens + ROWS - 1) / ROWS;
  const unsigned blocks = (unsigned)(needed < 1 << 16 ? needed : 1 << 16);
  const uint32_t lds = p.num_groups > 1 ? kRowsAtOnce * p.num_experts * 8u : 0u;
  if (!p.bias) pick_rows_kernel<V, VEC, kByLogits><<<blocks, kRowsAtOnce * 64, lds, stream>>>(p);
  else if (p.sigmoid) pick_rows_kernel<V, VEC, kBySigmoid><<<blocks, kRowsAtOnce * 64, lds, stream>>>(p);
  else pick_rows_kernel<V, VEC, kBySoftmax><<<blocks, kRowsAtOnce * 64, lds, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

// Four rows a wavefront for up to 512 experts without groups, or with groups
// that are whole lanes' runs of experts (16384 tokens of 256 experts in 8 groups
// 12.4 us, a row a wavefront in 64 bits 58.9); else a row a wavefront.
hipError_t launch_pick(const PickParams& p, hipStream_t stream) {
  if (p.num_tokens == 0) return hipSuccess;
  const int e = p.num_experts;
  if (e <= 512 && (p.num_groups == 1 || (e % 16 == 0 && 16 % p.num_groups == 0))) {
    if (e == 64) return launch_rows<4, true>(p, stream);
    if (e == 128) return launch_rows<8, true>(p, stream);
    if (e == 256) return launch_rows<16, true>(p, stream);
    if (e == 512) return launch_rows<32, true>(p, stream);
    if (e <= 64) return launch_rows<4, false>(p, stream);
    if (e <= 128) return launch_rows<8, false>(p, stream);
    if (e <= 192) return launch_rows<12, false>(p, stream);
    return e <= 256 ? launch_rows<16, false>(p, stream) : launch_rows<32, false>(p, stream);
  }
  if (e <= 64) return launch<1>(p, stream);
  if (e <= 128) return launch<2>(p, stream);
  if (e <= 256) return launch<4>(p, stream);
  if (e <= 512) return launch<8>(p, stream);
  if (e <= 1024) return launch<16>(p, stream);
  return launch<64>(p, stream);
}

}  // namespace llmoe
