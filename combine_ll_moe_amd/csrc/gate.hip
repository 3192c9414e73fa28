// The router's logits: hidden states times the experts' weights, in fp32.
//
// Mathematics: logits[t, e] = sum_c x[t, c] W[e, c], x in bf16. bf16 weights
// go through bf16 products, which are exact, with fp32 sums. An fp32 weight is
// cut into three bf16 parts of 8 bits each, W = W0 + W1 + W2 exactly, and
// three products share one fp32 sum: no bit of a weight is lost, where the
// matrix cores have no fp32 product of this rate. (A weight that is not finite
// has NaN for its rest; of a tiny one, bits below 2^-133, bf16's smallest, are
// left out, and a product sums subnormal values to some 17 bits.)
//
// Design, by how much work there is (launch_gate): a wavefront with one
// expert's row (gate_row_kernel); 16 tokens by a few experts, whose columns are
// split among the wavefronts (gate_few_kernel); tiles that come straight into
// LDS, steps ahead of the products (gate_tile_kernel).
//
// Bound: one token 3.5 us with bf16 weights (3.7 MB) and 128 tokens 6.7
// are latency: a launch, loads, and the sums' meeting. 16384 tokens (hidden 7168,
// 256 experts, bf16) take 78 to 83 us a launch, 720 to 770 TFLOP/s; their operands pass from the
// caches to LDS at 12 TB/s, and each SIMD's one or two wavefronts wait for each
// other at every step.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gate.h"
#include "tile.h"

namespace llmoe {
namespace {

constexpr int kColumns = 64;  // of a step
constexpr int kRowTokens = 4;
constexpr int64_t kFewLogits = 3 << 16, kFewLogitsFp32 = 1 << 18;
constexpr int64_t kCus = 256;

__device__ __forceinline__ uint32_t opaque_zero() {
  uint32_t zero = 0;
  asm volatile("" : "+v"(zero));
  return zero;
}

// Four fp32 in three bf16 parts of 8 bits, by cutting: the parts' signs and
// exponents are the value's own, so nothing overflows, and what is left after
// each cut is exact.
struct Parts4 {
  v2u part[3];
};
__device__ __forceinline__ Parts4 cut(v4u v) {
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  Parts4 o;
#pragma unroll
  for (int p = 0; p < 3; ++p) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      o.part[p][i] = __builtin_amdgcn_perm(__float_as_uint(f[2 * i + 1]), __float_as_uint(f[2 * i]), 0x07060302u);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] -= __uint_as_float(__float_as_uint(f[i]) & 0xFFFF0000u);
  }
  return o;
}
struct Parts {
  bf16x8 part[3];
};
__device__ __forceinline__ Parts cut(v4u a, v4u b) {
  const Parts4 x = cut(a), y = cut(b);
  Parts o;
#pragma unroll
  for (int p = 0; p < 3; ++p)
    o.part[p] = __builtin_bit_cast(bf16x8, v4u{x.part[p][0], x.part[p][1], y.part[p][0], y.part[p][1]});
  return o;
}

// A few tokens: a wavefront has one expert, every lane 8 columns at a time.
template <bool FP32, int T>
__global__ void __launch_bounds__(64) gate_row_kernel(const GateParams P) {
  constexpr int D = 8;  // loads of W under way
  const int lane = threadIdx.x, e = blockIdx.x;
  const uint32_t ldx = (uint32_t)P.hidden * 2, ldw = (uint32_t)P.hidden * (FP32 ? 4 : 2);
  const Rsrc rw = rsrc_of(P.w + (uint64_t)e * ldw, ldw);
  const Rsrc rx = rsrc_of(P.x, (uint32_t)P.num_tokens * ldx);
  const int steps = (P.hidden + 511) / 512;
  v4u wb[D][FP32 ? 2 : 1], xb[D][T];
  auto load = [&](int s, int step) {
    const uint32_t c = (uint32_t)step * 512 + lane * 8;
    const bool in = c < (uint32_t)P.hidden;
#pragma unroll
    for (int i = 0; i < (FP32 ? 2 : 1); ++i)
      wb[s][i] = __builtin_amdgcn_raw_buffer_load_b128(rw, (int)(in ? c * (FP32 ? 4 : 2) + 16 * i : kOutside), 0, 0);
#pragma unroll
    for (int t = 0; t < T; ++t)
      xb[s][t] = __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(in ? t * ldx + c * 2 : kOutside), 0, 0);
  };
  float sum[T] = {};
#pragma unroll
  for (int s = 0; s < D; ++s) load(s, s);
  for (int k = 0; k < steps; k += D) {
#pragma unroll
    for (int s = 0; s < D; ++s) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (FP32) {
          w[i] = __uint_as_float(wb[s][0][i]);
          w[4 + i] = __uint_as_float(wb[s][1][i]);
        } else {
          w[2 * i] = __uint_as_float(wb[s][0][i] << 16);
          w[2 * i + 1] = __uint_as_float(wb[s][0][i] & 0xFFFF0000u);
        }
      }
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[t] = __builtin_fmaf(__uint_as_float(xb[s][t][i] << 16), w[2 * i], sum[t]);
          sum[t] = __builtin_fmaf(__uint_as_float(xb[s][t][i] & 0xFFFF0000u), w[2 * i + 1], sum[t]);
        }
      load(s, k + s + D);
    }
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum[t] += __shfl_xor(sum[t], d, 64);
    if (lane == 0 && t < P.num_tokens) P.logits[(int64_t)t * P.num_experts + e] = sum[t];
  }
}

// 16 tokens x EW experts (as few as the GPU has room for). fp32 weights are
// cut on their way into LDS, once each (cut as fragments, whose 16 rows repeat
// the EW, 128 tokens by 256 experts took 11.2 us, cut once with loads two steps
// ahead 10.7, and one step ahead, as it is, 9.2: fewer registers, more wavefronts).
template <bool FP32, int EW, int WAVES>
__global__ void __launch_bounds__(WAVES * 64) gate_few_kernel(const GateParams P) {
  constexpr int ITEM = FP32 ? 4 : 2, WROW = kColumns * ITEM, WL = (EW * WROW + 1023) / 1024;
  constexpr int XPART = 16 * 128, PARTS = FP32 ? 3 : 1, WPART = PARTS * EW * 128;
  __shared__ __align__(16) uint8_t pool[WAVES * (XPART + WPART)];
  const int lane = threadIdx.x & 63, lo = lane & 15, hi = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int across = (P.num_experts + EW - 1) / EW, down = (P.num_tokens + 15) / 16;
  uint8_t* xl = pool + wave * (XPART + WPART);
  uint8_t* wl = xl + XPART;
  const uint32_t apart = opaque_zero();  // lanes read each other's rows
  const uint8_t* xr = xl + apart;
  const uint8_t* wr = wl + apart;
  const uint32_t ldx = (uint32_t)P.hidden * 2, ldw = (uint32_t)P.hidden * ITEM;
  const int steps = (P.hidden + kColumns - 1) / kColumns;
  const int s0 = steps * wave / WAVES, s1 = steps * (wave + 1) / WAVES;
  const int64_t tiles = (int64_t)across * down;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int e0 = (int)(t % across) * EW;
    const int64_t row0 = t / across * 16;
    const int rows = P.num_tokens - row0 < 16 ? (int)(P.num_tokens - row0) : 16;
    const int experts = P.num_experts - e0 < EW ? P.num_experts - e0 : EW;
    const Rsrc rx = rsrc_of(P.x + (uint64_t)row0 * ldx, (uint32_t)rows * ldx);
    const Rsrc rw = rsrc_of(P.w + (uint64_t)e0 * ldw, (uint32_t)experts * ldw);
    v4u xb[2], wb[WL];
    auto load = [&](int step) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t at = (uint32_t)step * 128 + (lane & 7) * 16;
        xb[i] = __builtin_amdgcn_raw_buffer_load_b128(
            rx, (int)(step < s1 && at < ldx ? ((lane >> 3) + 8 * i) * ldx + at : kOutside), 0, 0);
      }
#pragma unroll
      for (int i = 0; i < WL; ++i) {
        constexpr int CH = WROW / 16;
        const uint32_t at = (uint32_t)step * WROW + (lane % CH) * 16;
        wb[i] = __builtin_amdgcn_raw_buffer_load_b128(
            rw, (int)(step < s1 && at < ldw && lane / CH + 64 / CH * i < EW ? (lane / CH + 64 / CH * i) * ldw + at
                                                                             : kOutside),
            0, 0);
      }
    };
    auto store = [&] {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (lane >> 3) + 8 * i;
        *reinterpret_cast<v4u*>(xl + r * 128 + (((lane & 7) ^ r) & 7) * 16) = xb[i];
      }
#pragma unroll
      for (int i = 0; i < WL; ++i) {
        constexpr int CH = WROW / 16;
        const int r = lane / CH + 64 / CH * i, c = lane % CH;
        if (64 / CH > EW && r >= EW) continue;
        if constexpr (FP32) {
          const Parts4 v = cut(wb[i]);
#pragma unroll
          for (int p = 0; p < 3; ++p)
            *reinterpret_cast<v2u*>(wl + (p * EW + r) * 128 + ((c / 2 ^ r) & 7) * 16 + (c & 1) * 8) = v.part[p];
        } else {
          *reinterpret_cast<v4u*>(wl + r * 128 + ((c ^ r) & 7) * 16) = wb[i];
        }
      }
    };
    auto chunk = [&](const uint8_t* from, int r, int c) {
      return __builtin_bit_cast(bf16x8, *reinterpret_cast<const v4u*>(from + r * 128 + ((c ^ r) & 7) * 16));
    };
    const int wrow = lo & (EW - 1);
    f32x4 acc = {0, 0, 0, 0};
    auto multiply = [&] {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bf16x8 a = chunk(xr, lo, 4 * j + hi);
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(chunk(wr + p * EW * 128, wrow, 4 * j + hi), a, acc, 0, 0, 0);
      }
    };
    load(s0);
    for (int k = s0; k < s1; ++k) {
      store();
      load(k + 1);
      multiply();
    }
    // the wavefronts' sums meet: lane l holds experts 4 (l / 16) + r of token l % 16
    __syncthreads();
    float* sums = reinterpret_cast<float*>(pool);
    *reinterpret_cast<f32x4*>(sums + wave * 256 + lo * 16 + 4 * hi) = acc;
    __syncthreads();
    if (threadIdx.x < 256) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) v += sums[w * 256 + threadIdx.x];
      const int r = threadIdx.x / 16, e = threadIdx.x % 16;
      if (r < rows && e < experts) P.logits[(row0 + r) * P.num_experts + e0 + e] = v;
    }
    __syncthreads();
  }
}

// Many tokens: tiles of BM tokens x BN experts on WM x WN wavefronts, each FM
// x FN fragments; a step of 64 columns is copied straight into LDS, STAGES - 1
// steps ahead of the products.
template <bool FP32, int WM, int WN, int FM, int FN, int STAGES>
__global__ void __launch_bounds__(WM* WN * 64, 2) gate_tile_kernel(const GateParams P) {
  constexpr int BM = WM * FM * 16, BN = WN * FN * 16, WAVES = WM * WN;
  constexpr int ITEM = FP32 ? 4 : 2, WROW = kColumns * ITEM, CH = WROW / 16;
  constexpr int STAGE = BM * kStep + BN * WROW;
  constexpr int XC = BM / 8 / WAVES, WC = BN * WROW / 1024 / WAVES, LOADS = XC + WC;
  static_assert(STAGES >= 2 && STAGES <= 4 && BM / 8 % WAVES == 0 && BN * WROW / 1024 % WAVES == 0);
  // an array each, so that the compiler can tell a step's copies from the
  // reads of another one's
  __shared__ __align__(16) uint8_t st0[STAGE], st1[STAGE];
  __shared__ __align__(16) uint8_t st2[STAGES > 2 ? STAGE : 16], st3[STAGES > 3 ? STAGE : 16];
  const int tid = threadIdx.x, lane = tid & 63, lo = lane & 15, hi = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t ldx = (uint32_t)P.hidden * 2, ldw = (uint32_t)P.hidden * ITEM;
  const int steps = (P.hidden + kColumns - 1) / kColumns;
  const uint32_t across = (uint32_t)((P.num_experts + BN - 1) / BN);
  const uint32_t tile = run_of_xcd(blockIdx.x, gridDim.x);
  const int e0 = (int)(tile % across) * BN;
  const int64_t row0 = (int64_t)(tile / across) * BM;
  const int rows = P.num_tokens - row0 < BM ? (int)(P.num_tokens - row0) : BM;
  const int experts = P.num_experts - e0 < BN ? P.num_experts - e0 : BN;
  const Rsrc rx = rsrc_of(P.x + (uint64_t)row0 * ldx, (uint32_t)rows * ldx);
  const Rsrc rw = rsrc_of(P.w + (uint64_t)e0 * ldw, (uint32_t)experts * ldw);

  // A row's 16-byte chunks are permuted by the row's low bits, so that the 16
  // lanes that read one chunk of 16 rows meet no bank twice.
  const uint32_t xs = (uint32_t)lane >> 3, xc = ((lane & 7) ^ xs) * 16;
  constexpr int WR = 64 / CH;  // rows of W a copy
  const uint32_t ws = (uint32_t)lane / CH;
  auto fetch = [&](int step, uint8_t* lds) __attribute__((always_inline)) {
    const uint32_t from = (uint32_t)step * kStep + xc;
    const uint32_t at = step < steps && from < ldx ? xs * ldx + from : kOutside;
#pragma unroll
    for (int i = 0; i < XC; ++i) {
      const uint32_t g = i * WAVES + wave;
      copy16(rx, lds + g * 8 * kStep, at + g * 8 * ldx);
    }
#pragma unroll
    for (int i = 0; i < WC; ++i) {
      const uint32_t g = i * WAVES + wave, r = g * WR + ws;
      const uint32_t wfrom = (uint32_t)step * WROW + ((lane % CH) ^ (r & (CH - 1))) * 16;
      copy16(rw, lds + BM * kStep + g * 1024, step < steps && wfrom < ldw ? r * ldw + wfrom : kOutside);
    }
  };
  auto x_chunk = [&](const uint8_t* lds, int m, int c) {
    const int r = wm * FM * 16 + m * 16 + lo;
    return *reinterpret_cast<const v4u*>(lds + r * kStep + ((c ^ (r & 7)) << 4));
  };
  auto w_chunk = [&](const uint8_t* lds, int f, int c) {
    const int r = wn * FN * 16 + f * 16 + lo;
    return *reinterpret_cast<const v4u*>(lds + BM * kStep + r * WROW + ((c ^ (r & (CH - 1))) << 4));
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int f = 0; f < FN; ++f) acc[m][f] = f32x4{0, 0, 0, 0};
  auto multiply = [&](const uint8_t* lds) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      bf16x8 a[FM];
#pragma unroll
      for (int m = 0; m < FM; ++m) a[m] = __builtin_bit_cast(bf16x8, x_chunk(lds, m, 4 * j + hi));
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        if constexpr (FP32) {
          const Parts w = cut(w_chunk(lds, f, 8 * j + 2 * hi), w_chunk(lds, f, 8 * j + 2 * hi + 1));
#pragma unroll
          for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int m = 0; m < FM; ++m)
              acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.part[p], a[m], acc[m][f], 0, 0, 0);
        } else {
          const bf16x8 w = __builtin_bit_cast(bf16x8, w_chunk(lds, f, 4 * j + hi));
#pragma unroll
          for (int m = 0; m < FM; ++m)
            acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, a[m], acc[m][f], 0, 0, 0);
        }
      }
    }
  };
  constexpr int AHEAD = STAGES - 1;
  uint8_t* const buffers[4] = {st0, st1, st2, st3};
#pragma unroll
  for (int s = 0; s < AHEAD; ++s) fetch(s, buffers[s]);
  for (int k = 0; k < steps; k += STAGES) {
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      wait_loads<(AHEAD - 1) * LOADS>();
      meet();
      fetch(k + s + AHEAD, buffers[(s + AHEAD) % STAGES]);
      __builtin_amdgcn_sched_barrier(0);
      multiply(buffers[s]);
    }
  }
  wait_loads<0>();  // no copy is under way when the LDS is another workgroup's
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const int r = wm * FM * 16 + m * 16 + lo;
    if (r >= rows) continue;
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      const int e = wn * FN * 16 + f * 16 + 4 * hi;
      float* to = P.logits + (row0 + r) * P.num_experts + e0 + e;
      if (P.num_experts % 4 == 0) {
        if (e < experts) *reinterpret_cast<f32x4*>(to) = acc[m][f];
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (e + q < experts) to[q] = acc[m][f][q];
      }
    }
  }
}

template <bool FP32, int WM, int WN, int FM, int FN, int STAGES>
hipError_t launch_tile(const GateParams& p, hipStream_t stream) {
  constexpr int BM = WM * FM * 16, BN = WN * FN * 16, THREADS = WM * WN * 64;
  const int64_t across = (p.num_experts + BN - 1) / BN;
  // a grid has fewer than 2^32 threads: more rows go out in several launches
  const int64_t most = (1ll << 31) / THREADS / across * BM;
  GateParams q = p;
  for (int64_t first = 0; first < p.num_tokens; first += most) {
    q.x = p.x + (uint64_t)first * p.hidden * 2;
    q.logits = p.logits + first * p.num_experts;
    q.num_tokens = (int)(p.num_tokens - first < most ? p.num_tokens - first : most);
    const int64_t tiles = across * ((q.num_tokens + (int64_t)BM - 1) / BM);
    gate_tile_kernel<FP32, WM, WN, FM, FN, STAGES><<<(unsigned)tiles, THREADS, 0, stream>>>(q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool FP32, int EW, int WAVES>
hipError_t launch_few(const GateParams& p, hipStream_t stream) {
  const int64_t tiles = (((int64_t)p.num_tokens + 15) / 16) * ((p.num_experts + EW - 1) / EW);
  const unsigned blocks = (unsigned)(tiles < 1 << 16 ? tiles : 1 << 16);
  gate_few_kernel<FP32, EW, WAVES><<<blocks, WAVES * 64, 0, stream>>>(p);
  return hipGetLastError();
}

template <bool FP32>
hipError_t launch_row(const GateParams& p, hipStream_t stream) {
  if (p.num_tokens == 1) gate_row_kernel<FP32, 1><<<p.num_experts, 64, 0, stream>>>(p);
  else if (p.num_tokens == 2) gate_row_kernel<FP32, 2><<<p.num_experts, 64, 0, stream>>>(p);
  else gate_row_kernel<FP32, 4><<<p.num_experts, 64, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

// Which kernel, by the sizes (us a launch in a row of launches, operands out of the
// caches, all at hidden 7168 and 256 experts, weights bf16 | fp32). Up to kRowTokens
// tokens: a wavefront an expert (1 token 3.5 | 4.2, where 16 x 8 take 6.0 | 9.6; 4 tokens
// 6.1 | 6.5 against 6.0 | 9.8). Then 16 tokens by as few experts as fill the GPU once, 4
// with fp32 weights alone (64 tokens: 16 x 4
// 6.3 | 8.2, 16 x 8 6.4 | 8.9, 16 x 16 7.7 | 11.2; 128 tokens 10.4 | 13.5, 6.7 | 9.2, 7.9 |
// 11.4; 256 tokens 16 x 16 8.4 | 12.1), more than 256 of those with eight wavefronts (512
// tokens 13.2 | 21.6, with sixteen 13.7 | 22.4), up to as many logits as tiles do faster
// (768 tokens 18.7 against 21.3, 1024 tokens 27 against 24 | 44 against 48). Then the
// smallest tiles that are not too many: 64 x 32 (2048 tokens 30 | 51, in 64 x 64 34 | 79; 4096 tokens 50 |
// 77), then with bf16 64 x 64 (4096 tokens 36; 8192 63), 64 x 128, two a CU (4096
// tokens 52, 8192 54, 10000 96), and 128 x 128 (8192 tokens 70, 10000 71, 16384
// 78), with fp32 128 x 32 (4096 tokens 93, 8192 110, 16384 216) and 128 x 64
// (8192 tokens 118, 16384 193).
hipError_t launch_gate(const GateParams& p, hipStream_t stream) {
  if (p.num_tokens == 0) return hipSuccess;
  auto tiles = [&](int64_t tokens, int64_t experts) {
    return (p.num_tokens + tokens - 1) / tokens * ((p.num_experts + experts - 1) / experts);
  };
  if (p.num_tokens <= kRowTokens) return p.w_fp32 ? launch_row<true>(p, stream) : launch_row<false>(p, stream);
  const int64_t logits = (int64_t)p.num_tokens * p.num_experts;
  if (p.w_fp32) {
    if (logits <= kFewLogitsFp32) {
      if (tiles(16, 4) <= kCus) return launch_few<true, 4, 16>(p, stream);
      if (tiles(16, 8) <= kCus) return launch_few<true, 8, 16>(p, stream);
      return tiles(16, 16) <= kCus ? launch_few<true, 16, 16>(p, stream) : launch_few<true, 16, 8>(p, stream);
    }
    if (tiles(64, 32) <= 2 * kCus) return launch_tile<true, 2, 2, 2, 1, 4>(p, stream);
    return tiles(128, 64) < 2 * kCus ? launch_tile<true, 2, 2, 4, 1, 2>(p, stream)
                                     : launch_tile<true, 2, 2, 4, 2, 2>(p, stream);
  }
  if (logits <= kFewLogits) {
    if (tiles(16, 8) <= kCus) return launch_few<false, 8, 16>(p, stream);
    return tiles(16, 16) <= kCus ? launch_few<false, 16, 16>(p, stream) : launch_few<false, 16, 8>(p, stream);
  }
  if (tiles(64, 32) <= kCus) return launch_tile<false, 2, 2, 2, 1, 4>(p, stream);
  if (tiles(64, 64) <= kCus) return launch_tile<false, 2, 2, 2, 2, 4>(p, stream);
  return tiles(64, 128) <= kCus ? launch_tile<false, 4, 2, 1, 4, 3>(p, stream)
                                : launch_tile<false, 2, 4, 4, 2, 4>(p, stream);
}

}  // namespace llmoe
