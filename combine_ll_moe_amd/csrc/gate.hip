// The router's logits: hidden states times the experts' weights, in fp32.
//
// Mathematics: logits[t, e] = sum_c x[t, c] W[e, c], x in bf16. bf16 weights
// go through bf16 products, which are exact, with fp32 sums. An fp32 weight is
// cut into three bf16 parts of 8 bits each, W = W0 + W1 + W2 exactly, and
// three products share one fp32 sum: no bit of a weight is lost, where the
// matrix cores have no fp32 product of this rate. (A weight that is not finite
// has NaN for its rest.)
//
// Design: a workgroup has 16 tokens x 16 experts; its eight wavefronts split
// the columns and add up through LDS. Rows come by whole lines into
// registers, some steps ahead, and through LDS into the products' order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_gemm.h"
#include "gate.h"

namespace llmoe {
namespace {

constexpr int kWaves = 8;
constexpr int kColumns = 64;  // of a step

__device__ __forceinline__ uint32_t opaque_zero() {
  uint32_t zero = 0;
  asm volatile("" : "+v"(zero));
  return zero;
}

// Eight fp32 in three bf16 parts of 8 bits, by cutting: the parts' signs and
// exponents are the value's own, so nothing overflows, and what is left after
// each cut is exact.
struct Parts {
  bf16x8 part[3];
};
__device__ __forceinline__ Parts cut(v4u a, v4u b) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = __uint_as_float(a[i]);
    f[4 + i] = __uint_as_float(b[i]);
  }
  Parts o;
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    v4u packed;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      packed[i] = __builtin_amdgcn_perm(__float_as_uint(f[2 * i + 1]), __float_as_uint(f[2 * i]), 0x07060302u);
    o.part[p] = __builtin_bit_cast(bf16x8, packed);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] -= __uint_as_float(__float_as_uint(f[i]) & 0xFFFF0000u);
  }
  return o;
}

template <bool FP32>
__global__ void __launch_bounds__(kWaves * 64) gate_few_kernel(const GateParams P) {
  constexpr int ITEM = FP32 ? 4 : 2, WROW = kColumns * ITEM, WL = FP32 ? 4 : 2, D = 4;
  constexpr int XPART = 16 * 128, WPART = 16 * WROW;
  __shared__ __align__(16) uint8_t pool[kWaves * (XPART + WPART)];
  const int lane = threadIdx.x & 63, lo = lane & 15, hi = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int across = (P.num_experts + 15) / 16, down = (P.num_tokens + 15) / 16;
  uint8_t* xl = pool + wave * (XPART + WPART);
  uint8_t* wl = xl + XPART;
  const uint32_t apart = opaque_zero();  // lanes read each other's rows
  const uint8_t* xr = xl + apart;
  const uint8_t* wr = wl + apart;
  const uint32_t ldx = (uint32_t)P.hidden * 2, ldw = (uint32_t)P.hidden * ITEM;
  const int steps = (P.hidden + kColumns - 1) / kColumns;
  const int s0 = steps * wave / kWaves, s1 = steps * (wave + 1) / kWaves;
  const int64_t tiles = (int64_t)across * down;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int e0 = (int)(t % across) * 16;
    const int64_t row0 = t / across * 16;
    const int rows = P.num_tokens - row0 < 16 ? (int)(P.num_tokens - row0) : 16;
    const int experts = P.num_experts - e0 < 16 ? P.num_experts - e0 : 16;
    const Rsrc rx = rsrc_of(P.x + (uint64_t)row0 * ldx, (uint32_t)rows * ldx);
    const Rsrc rw = rsrc_of(P.w + (uint64_t)e0 * ldw, (uint32_t)experts * ldw);
    v4u xb[D][2], wb[D][WL];
    auto load = [&](int s, int step) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t at = (uint32_t)step * 128 + (lane & 7) * 16;
        xb[s][i] = __builtin_amdgcn_raw_buffer_load_b128(
            rx, (int)(step < s1 && at < ldx ? ((lane >> 3) + 8 * i) * ldx + at : kOutside), 0, 0);
      }
#pragma unroll
      for (int i = 0; i < WL; ++i) {
        constexpr int CH = WROW / 16;
        const uint32_t at = (uint32_t)step * WROW + (lane % CH) * 16;
        wb[s][i] = __builtin_amdgcn_raw_buffer_load_b128(
            rw, (int)(step < s1 && at < ldw ? (lane / CH + 64 / CH * i) * ldw + at : kOutside), 0, 0);
      }
    };
    auto store = [&](int s) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (lane >> 3) + 8 * i;
        *reinterpret_cast<v4u*>(xl + r * 128 + (((lane & 7) ^ r) & 7) * 16) = xb[s][i];
      }
#pragma unroll
      for (int i = 0; i < WL; ++i) {
        constexpr int CH = WROW / 16;
        const int r = lane / CH + 64 / CH * i, c = lane % CH;
        *reinterpret_cast<v4u*>(wl + r * WROW + ((c ^ r) & (CH - 1)) * 16) = wb[s][i];
      }
    };
    auto chunk = [&](const uint8_t* from, int row_bytes, int c) {
      return *reinterpret_cast<const v4u*>(from + lo * row_bytes + ((c ^ lo) & (row_bytes / 16 - 1)) * 16);
    };
    f32x4 acc = {0, 0, 0, 0};
    auto multiply = [&] {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bf16x8 a = __builtin_bit_cast(bf16x8, chunk(xr, 128, 4 * j + hi));
        if constexpr (FP32) {
          const Parts w = cut(chunk(wr, WROW, 8 * j + 2 * hi), chunk(wr, WROW, 8 * j + 2 * hi + 1));
#pragma unroll
          for (int p = 0; p < 3; ++p) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.part[p], a, acc, 0, 0, 0);
        } else {
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, chunk(wr, WROW, 4 * j + hi)), a, acc,
                                                       0, 0, 0);
        }
      }
    };
#pragma unroll
    for (int s = 0; s < D; ++s) load(s, s0 + s);
    for (int k = s0; k < s1; k += D) {
#pragma unroll
      for (int s = 0; s < D; ++s) {
        if (k + s < s1) {
          store(s);
          load(s, k + s + D);
          multiply();
        }
      }
    }
    // the wavefronts' sums meet: lane l holds experts 4 (l / 16) + r of token l % 16
    __syncthreads();
    float* sums = reinterpret_cast<float*>(pool);
    *reinterpret_cast<f32x4*>(sums + wave * 256 + lo * 16 + 4 * hi) = acc;
    __syncthreads();
    if (threadIdx.x < 256) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += sums[w * 256 + threadIdx.x];
      const int r = threadIdx.x / 16, e = threadIdx.x % 16;
      if (r < rows && e < experts) P.logits[(row0 + r) * P.num_experts + e0 + e] = v;
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_gate(const GateParams& p, hipStream_t stream) {
  if (p.num_tokens == 0) return hipSuccess;
  const int64_t tiles = (((int64_t)p.num_tokens + 15) / 16) * ((p.num_experts + 15) / 16);
  const unsigned blocks = (unsigned)(tiles < 1 << 16 ? tiles : 1 << 16);
  if (p.w_fp32) gate_few_kernel<true><<<blocks, kWaves * 64, 0, stream>>>(p);
  else gate_few_kernel<false><<<blocks, kWaves * 64, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace llmoe
