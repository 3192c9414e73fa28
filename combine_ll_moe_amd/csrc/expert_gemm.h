// Products grouped by expert: what the kernels and the C ABI share.
//
// Expert e owns rows [e * max_tokens, (e + 1) * max_tokens) of the activations
// and of the output and fills the first counts[e] of them, as the dispatch's
// expert side leaves them. P = A W_e^T over those rows; the gated form takes
// W_e of 2n rows and gives silu(P[:, :n]) * P[:, n:].
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace llmoe {

enum : int { kWeightBf16 = 0, kWeightFp8 = 1, kWeightInt4 = 2 };

struct GemmParams {
  const uint8_t* a;         // bf16 or e4m3 [num_experts * max_tokens, k]
  const float* a_scales;    // fp8: [num_experts * max_tokens, k / 128]
  const uint8_t* w;         // [num_experts, n or 2n, k]; int4: k / 2 bytes a row
  const void* w_scales;     // fp8: fp32 per 128 x 128; int4: bf16 per row and group
  const uint8_t* w_zeros;   // int4: zero points as the scales, or null (8)
  const int32_t* counts;    // [num_experts]
  uint8_t* out;             // bf16 or e4m3 [num_experts * max_tokens, n]
  float* out_scales;        // fp8 out: [num_experts * max_tokens, n / 128]
  int max_tokens;
  int num_experts;
  int n;                    // output columns
  int k;
  int group;                // int4: weights along k that share a scale
  int weight;               // kWeight...
  int gated;                // silu(gate) * up
  int out_fp8;
};

// LDS of the tile prefix below: a word an expert and the total, then the
// experts' rows (up to kRowsKept experts; the tiles' buffers leave no more).
constexpr int kRowsKept = 2048;
inline uint32_t tile_prefix_bytes(int num_experts) {
  return ((uint32_t)(num_experts + 1 + (num_experts <= kRowsKept ? num_experts : 0)) * 4u + 15u) & ~15u;
}

// Who takes which rows. An expert with at most `most` rows is the few kernel's,
// in tiles of kFewRows; of one with more the tile kernel takes tiles of
// kTileRows, and the few kernel the rows behind the last whole one if they
// fit in one of its own.
constexpr int kFewRows = 64;
constexpr int kTileRows = 256;
__host__ __device__ __forceinline__ int few_first(int rows, int most) {
  return rows <= most ? 0 : rows - rows % kTileRows;
}
__host__ __device__ __forceinline__ int few_rows(int rows, int most) {
  if (rows <= 0) return 0;
  if (rows <= most) return rows;
  const int left = rows % kTileRows;
  return left <= kFewRows ? left : 0;
}
// What a strip of W costs the few kernel with a tile of so many rows, in
// eighths of one with up to 16 (measured, us for 64 experts of 2048 x 7168
// weights at 16, 32 and 64 rows: bf16 314, 314, 331; fp8 169, 183, 203; int4
// 107, 140, 210).
template <int WEIGHT>
__device__ __forceinline__ int strip_cost(int rows) {
  if (WEIGHT == kWeightBf16) return rows <= 32 ? 8 : 9;
  if (WEIGHT == kWeightFp8) return rows <= 16 ? 8 : rows <= 32 ? 9 : 10;
  return rows <= 16 ? 8 : rows <= 32 ? 10 : 16;
}
// The same of all row tiles of few_rows rows.
template <int WEIGHT>
__device__ __forceinline__ int tiles_cost(int rows) {
  const int whole = rows / kFewRows, left = rows % kFewRows;
  return whole * strip_cost<WEIGHT>(kFewRows) + (left ? strip_cost<WEIGHT>(left) : 0);
}
__host__ __device__ __forceinline__ int big_tiles(int rows, int most) {
  return rows <= most ? 0 : rows / kTileRows + (rows % kTileRows > kFewRows);
}

// Inclusive sums over a wavefront's lanes, in DPP steps (by 1, 2, 4, 8 lanes
// within rows of 16, then the rows' totals): a few cycles each, where a step
// through LDS takes a hundred.
template <int CTRL, int ROWS, int BANKS>
__device__ __forceinline__ uint32_t dpp_add(uint32_t v) {
  return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, BANKS, false);
}
__device__ __forceinline__ uint32_t wave_sums(uint32_t v) {
  v = dpp_add<0x111, 0xF, 0xF>(v);  // row_shr:1
  v = dpp_add<0x112, 0xF, 0xF>(v);  // row_shr:2
  v = dpp_add<0x114, 0xF, 0xE>(v);  // row_shr:4
  v = dpp_add<0x118, 0xF, 0xC>(v);  // row_shr:8
  v = dpp_add<0x142, 0xA, 0xF>(v);  // row_bcast:15
  return dpp_add<0x143, 0xC, 0xF>(v);  // row_bcast:31
}

// What stands before each expert: pre[e], e <= E, of measure(rows), such as
// its row tiles; the rows of each expert behind them (kRowsKept). All THREADS threads
// call it; scan: one word a wavefront.
template <int THREADS, class Measure>
__device__ __forceinline__ void tile_prefix(const GemmParams& P, uint32_t* pre, uint32_t* scan,
                                            Measure measure) {
  const int tid = threadIdx.x, lane = tid & 63, E = P.num_experts;
  const int run = (E + THREADS - 1) / THREADS;
  const int e0 = tid * run < E ? tid * run : E, e1 = e0 + run < E ? e0 + run : E;
  uint32_t sum = 0;
  for (int e = e0; e < e1; ++e) {
    int c = P.counts[e];
    c = c < P.max_tokens ? c : P.max_tokens;
    const uint32_t t = (uint32_t)measure(c);
    pre[e] = sum;
    if (E <= kRowsKept) pre[E + 1 + e] = (uint32_t)c;
    sum += t;
  }
  const uint32_t incl = wave_sums(sum);
  if (lane == 63) scan[tid / 64] = incl;
  __syncthreads();
  uint32_t base = incl - sum;
  for (int w = 0; w < tid / 64; ++w) base += scan[w];
  for (int e = e0; e < e1; ++e) pre[e] += base;
  if (tid == THREADS - 1) pre[E] = base + sum;
  __syncthreads();
}

// Rows of expert e (the same for the whole workgroup).
__device__ __forceinline__ int rows_of(const GemmParams& P, const uint32_t* pre, int e) {
  int c;
  if (P.num_experts <= kRowsKept) {
    c = (int)pre[P.num_experts + 1 + e];
  } else {
    c = P.counts[e];
    c = c < P.max_tokens ? c : P.max_tokens;
  }
  return __builtin_amdgcn_readfirstlane(c);
}

// Expert of tile t < pre[E]: as many as have their last tile before t. All
// lanes of a wavefront look, 64 experts at a time (E <= 4096: at most twice);
// the answer is the same for all.
__device__ __forceinline__ int expert_of_tile(const uint32_t* pre, int E, uint32_t t) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  if (E > 64) {
    const int run = (E + 63) / 64, last = (lane + 1) * run;
    base = run * __popcll(__ballot(last < E && pre[last < E ? last : E] <= t));
  }
  const int e = base + lane;
  return base + __popcll(__ballot(e < E && pre[e < E ? e + 1 : E] <= t));
}

typedef __amdgpu_buffer_rsrc_t Rsrc;
constexpr uint32_t kOutside = 0x7FFFFFF0u;  // an offset behind every descriptor's range
__device__ __forceinline__ Rsrc rsrc_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, kBufferWord3);
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// fp32 -> bf16, nearest even, two at a time (gfx950's conversion
// instruction; NaN stays NaN).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

// 16 e4m3 codes as bf16, which holds them exactly.
struct Bf16x16 {
  bf16x8 lo, hi;
};
__device__ __forceinline__ Bf16x16 fp8_to_bf16(v4u v) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __builtin_bit_cast(
        uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, false));
    o[2 * i + 1] = __builtin_bit_cast(
        uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, true));
  }
  return {__builtin_bit_cast(bf16x8, v4u{o[0], o[1], o[2], o[3]}),
          __builtin_bit_cast(bf16x8, v4u{o[4], o[5], o[6], o[7]})};
}

// Eight codes of a word as bf16 16 + c, in the order 0 4 1 5 2 6 3 7. The two
// constants come in registers: an and-or takes no literals, and with literals
// each would be two instructions.
struct CodeMasks {
  uint32_t keep, base;
  __device__ CodeMasks() : keep(0x00780078u), base(0x41804180u) {
    asm("" : "+s"(keep), "+v"(base));
  }
};
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t w, const CodeMasks& c) {
  const v4u v = {((w << 3) & c.keep) | c.base, ((w >> 1) & c.keep) | c.base,
                 ((w >> 5) & c.keep) | c.base, ((w >> 9) & c.keep) | c.base};
  return __builtin_bit_cast(bf16x8, v);
}
// Eight bf16 of A in that order.
__device__ __forceinline__ bf16x8 a_like_codes(v4u a) {
  const v4u v = {__builtin_amdgcn_perm(a.z, a.x, 0x05040100u), __builtin_amdgcn_perm(a.z, a.x, 0x07060302u),
                 __builtin_amdgcn_perm(a.w, a.y, 0x05040100u), __builtin_amdgcn_perm(a.w, a.y, 0x07060302u)};
  return __builtin_bit_cast(bf16x8, v);
}

// silu(g) * u in fp32. exp(-g) overflows to infinity for g below about -88:
// the quotient is then -0, which is silu's limit.
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g / (1.0f + __expf(-g)) * u;
}

// Scale of 128 columns with largest magnitude amax, and what they are
// multiplied by for their codes: amax / 448 and 448 / amax, as the dispatch
// quantizes, but no scale below 2^-127: there 448 / amax would be infinite,
// and a zero's code NaN (a row whose gates all lie below -86 has such values).
struct BlockScale {
  float scale, inv;
};
__device__ __forceinline__ BlockScale block_scale(float amax) {
  if (!(amax > 0.0f)) return {0.0f, 0.0f};
  return {fmaxf(amax / 448.0f, 0x1p-127f), fminf(448.0f / amax, 0x1p127f)};
}

// fp32 -> OCP e4m3 codes, four packed little-endian: nearest even, +-448 for
// everything beyond and for the infinities, 0x7F for NaN. (As the dispatch's
// encoder, without its branch around the NaN's patch.)
__device__ __forceinline__ uint32_t e4m3_pack4(float p0, float p1, float p2, float p3) {
  const float c0 = __builtin_amdgcn_fmed3f(p0, -448.0f, 448.0f);
  const float c1 = __builtin_amdgcn_fmed3f(p1, -448.0f, 448.0f);
  const float c2 = __builtin_amdgcn_fmed3f(p2, -448.0f, 448.0f);
  const float c3 = __builtin_amdgcn_fmed3f(p3, -448.0f, 448.0f);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(c0, c1, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c2, c3, w, true);
  const uint32_t m = (p0 != p0 ? 0xFFu : 0u) | (p1 != p1 ? 0xFF00u : 0u) |
                     (p2 != p2 ? 0xFF0000u : 0u) | (p3 != p3 ? 0xFF000000u : 0u);
  return ((uint32_t)w & ~m) | (0x7F7F7F7Fu & m);
}

// Each takes its rows of every expert (few_rows, big_tiles).
hipError_t launch_gemm_few(const GemmParams& p, int most, hipStream_t stream);
hipError_t launch_gemm_few_fp8(const GemmParams& p, int most, hipStream_t stream);
hipError_t launch_gemm_few_int4(const GemmParams& p, int most, hipStream_t stream);
hipError_t launch_gemm_tile(const GemmParams& p, int most, hipStream_t stream);

}  // namespace llmoe
