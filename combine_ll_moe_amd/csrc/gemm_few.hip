// Products grouped by expert, for experts with few rows: every weight is read
// once from HBM and used for at most 64 rows, so the weights' bytes bound it.
//
// Mathematics: P[r, i] = sum_k A[r, k] W[i, k] for the rows of one expert, in
// 16-row fragments of A and 16-row strips of W on the matrix cores.
//   bf16: 16x16x32 products summed in fp32.
//   fp8:  codes become bf16, which holds them exactly, on their way to the
//         same products; the sum of 128 columns is scaled by the activation's
//         and the weight's scale and added up in fp32. (The matrix cores' own
//         fp8 products keep a sum to about 6e-6 of its magnitudes, and here
//         there is time to spare.)
//   int4: W = s (c - z), c the code, z the zero point, s the group's scale.
//         With c' = 16 + c, which bf16 holds exactly as 0x4180 | c << 3,
//         sum x W = s (sum x c' - (16 + z) sum x): codes become bf16 with a
//         shift and an and-or for every two, and no weight is rounded. sum x
//         is one more matrix product, with ones, shared by all strips.
//
// Design: a wavefront reads its fragments of W straight from memory into
// registers, several chunks of k ahead; no LDS copy, no barrier inside the k
// loop. Rows of A behind the expert's count, rows of W behind n and columns
// behind k are beyond their buffer descriptors' range: those loads return
// zeros and touch no memory. The strips of all experts form one list that is
// dealt in equal runs, so experts of any count and calls of any number of
// experts fill the GPU alike: to wavefronts, each alone with four strips over
// all of k, where the list is long; to workgroups whose wavefronts split k and
// add their sums up in LDS, where it is short.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_gemm.h"
#include "kernels.h"

namespace llmoe {
namespace {

typedef __amdgpu_buffer_rsrc_t Rsrc;
constexpr uint32_t kOutside = 0x7FFFFFF0u;  // an offset behind every descriptor's range
constexpr int kFewRows = 64;      // rows of a tile
constexpr int kFewFrags = 4;      // weight strips a wavefront holds at once
constexpr int kPartLd = kFewFrags * 16 + 4;  // floats of a row of partial sums, at most

__device__ __forceinline__ Rsrc rsrc_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, kBufferWord3);
}
__device__ __forceinline__ v4u load16(Rsrc r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
}

// One 16-row strip list of one expert and row tile.
struct Item {
  const uint8_t* a;       // first row of the tile
  const float* a_scales;
  int64_t row0;           // first output row
  int rows;               // filled rows of the tile
  int e;
  int strip;              // first output strip (16 columns)
  int strips;             // output strips to do
};

// Weight rows of fragment f of an item: the output strips in order, gated:
// first their gate rows, then their up rows.
template <int NF, bool GATED>
__device__ __forceinline__ int strip_row(const GemmParams& P, int strip, int f) {
  if constexpr (GATED)
    return (f < NF / 2 ? 0 : P.n) + 16 * (strip + (f < NF / 2 ? f : f - NF / 2));
  else
    return 16 * (strip + f);
}
// Filled rows of that strip (0 behind the item's strips).
template <int NF, bool GATED>
__device__ __forceinline__ int strip_rows(const GemmParams& P, const Item& it, int f) {
  const int s = GATED && f >= NF / 2 ? f - NF / 2 : f;
  if (s >= it.strips) return 0;
  const int left = P.n - 16 * (it.strip + s);
  return left < 16 ? left : 16;
}

// acc[mf][nf]: bf16 and int4: lane l holds rows 4 (l / 16) + r, r < 4, of
// column l % 16; fp8: columns 4 (l / 16) + r of row l % 16.
template <int MF, int NF, bool GATED>
__device__ __forceinline__ void sum_bf16(const GemmParams& P, const Item& it, int kw, int WK,
                                         f32x4 (&acc)[MF][NF]) {
  constexpr int D = MF == 4 ? 2 : 3;  // chunks in flight
  const int lane = threadIdx.x & 63;
  const uint32_t ld = 2u * (uint32_t)P.k;
  const Rsrc ra = rsrc_of(it.a, (uint32_t)it.rows * ld);
  Rsrc rw[NF];
  const uint8_t* w = P.w + (uint64_t)it.e * (GATED ? 2 : 1) * P.n * ld;
#pragma unroll
  for (int f = 0; f < NF; ++f)
    rw[f] = rsrc_of(w + (uint64_t)strip_row<NF, GATED>(P, it.strip, f) * ld,
                    (uint32_t)strip_rows<NF, GATED>(P, it, f) * ld);
  const uint32_t row = (lane & 15) * ld, col = 16u * (lane >> 4);
  const int chunks = (P.k + 63) / 64;
  v4u wb[D][NF][2], ab[D][MF][2];
  auto load = [&](int s, int c) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t at = 128u * (uint32_t)c + 64u * j + col;
      const bool in = c < chunks && at < ld;
      const uint32_t off = in ? row + at : kOutside;
#pragma unroll
      for (int f = 0; f < NF; ++f) wb[s][f][j] = load16(rw[f], off);
#pragma unroll
      for (int m = 0; m < MF; ++m) ab[s][m][j] = load16(ra, in ? off + m * 16u * ld : kOutside);
    }
  };
#pragma unroll
  for (int s = 0; s < D; ++s) load(s, kw + s * WK);
  for (int c = kw; c < chunks; c += D * WK) {
#pragma unroll
    for (int s = 0; s < D; ++s) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
          for (int f = 0; f < NF; ++f)
            acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, ab[s][m][j]), __builtin_bit_cast(bf16x8, wb[s][f][j]),
                acc[m][f], 0, 0, 0);
      load(s, c + (s + D) * WK);
    }
  }
}

template <int MF, int NF, bool GATED>
__device__ __forceinline__ void sum_fp8(const GemmParams& P, const Item& it, int kw, int WK,
                                        f32x4 (&acc)[MF][NF]) {
  constexpr int D = MF == 4 ? 1 : MF == 2 ? 2 : 3;
  const int lane = threadIdx.x & 63, lo = lane & 15, hi = lane >> 4;
  const uint32_t ld = (uint32_t)P.k;
  const int chunks = P.k / 128;
  const Rsrc ra = rsrc_of(it.a, (uint32_t)it.rows * ld);
  Rsrc rw[NF];
  const int rows_w = (GATED ? 2 : 1) * P.n, blocks = (rows_w + 127) / 128;
  const uint8_t* w = P.w + (uint64_t)it.e * rows_w * ld;
#pragma unroll
  for (int f = 0; f < NF; ++f)
    rw[f] = rsrc_of(w + (uint64_t)strip_row<NF, GATED>(P, it.strip, f) * ld,
                    (uint32_t)strip_rows<NF, GATED>(P, it, f) * ld);
  // Scales: lane quarter q loads row fragment q's (lane's row) and strip q's.
  const int arow = (MF > 1 ? hi % MF : 0) * 16 + lo;
  const float* as_p = it.a_scales + (uint64_t)(arow < it.rows ? arow : it.rows - 1) * chunks;
  const int wblock = strip_row<NF, GATED>(P, it.strip, hi % NF) / 128;
  const float* ws_p = static_cast<const float*>(P.w_scales) +
                      ((uint64_t)it.e * blocks + (wblock < blocks ? wblock : blocks - 1)) * chunks;
  const uint32_t row = lo * ld, col = 16u * hi;
  v4u wb[D][NF][2], ab[D][MF][2];
  float as[D], sw[D];
  auto load = [&](int s, int c) {
    const bool in = c < chunks;
    const uint32_t off = in ? row + 128u * (uint32_t)c + col : kOutside;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int f = 0; f < NF; ++f) wb[s][f][j] = load16(rw[f], off + 64u * j);
#pragma unroll
      for (int m = 0; m < MF; ++m) ab[s][m][j] = load16(ra, in ? off + 64u * j + m * 16u * ld : kOutside);
    }
    as[s] = as_p[in ? c : chunks - 1];  // a chunk behind k is zeros: any scale does
    sw[s] = ws_p[in ? c : chunks - 1];
  };
#pragma unroll
  for (int s = 0; s < D; ++s) load(s, kw + s * WK);
  for (int c = kw; c < chunks; c += D * WK) {
#pragma unroll
    for (int s = 0; s < D; ++s) {
      f32x4 p[MF][NF];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        Bf16x16 a[MF];
#pragma unroll
        for (int m = 0; m < MF; ++m) a[m] = fp8_to_bf16(ab[s][m][j]);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          const Bf16x16 wv = fp8_to_bf16(wb[s][f][j]);
#pragma unroll
          for (int m = 0; m < MF; ++m) {
            const f32x4 zero = {0, 0, 0, 0};
            p[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv.lo, a[m].lo, j ? p[m][f] : zero, 0, 0, 0);
            p[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv.hi, a[m].hi, p[m][f], 0, 0, 0);
          }
        }
      }
      const bool in = c + s * WK < chunks;  // else 0 * a scale that may be NaN
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        const float av = MF > 1 ? __shfl(as[s], m * 16 + lo, 64) : as[s];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          const float wv = __builtin_bit_cast(
              float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sw[s]), f * 16));
          const float sc = in ? av * wv : 0.0f;
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][f][r] = __builtin_fmaf(sc, p[m][f][r], acc[m][f][r]);
        }
      }
      load(s, c + (s + D) * WK);
    }
  }
}

// Eight codes of a word as bf16 16 + c, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t w) {
  const v4u v = {((w << 3) & 0x00780078u) | 0x41804180u, ((w >> 1) & 0x00780078u) | 0x41804180u,
                 ((w >> 5) & 0x00780078u) | 0x41804180u, ((w >> 9) & 0x00780078u) | 0x41804180u};
  return __builtin_bit_cast(bf16x8, v);
}
// Eight bf16 of A in that order.
__device__ __forceinline__ bf16x8 a_like_codes(v4u a) {
  const v4u v = {__builtin_amdgcn_perm(a.z, a.x, 0x05040100u), __builtin_amdgcn_perm(a.z, a.x, 0x07060302u),
                 __builtin_amdgcn_perm(a.w, a.y, 0x05040100u), __builtin_amdgcn_perm(a.w, a.y, 0x07060302u)};
  return __builtin_bit_cast(bf16x8, v);
}

// G / 32 products of 32 columns cover a group; lane quarter g holds columns
// [g G / 4, (g + 1) G / 4) of it, so that its codes are G / 8 bytes in a row.
template <int MF, int NF, bool GATED, int G>
__device__ __forceinline__ void sum_int4(const GemmParams& P, const Item& it, int kw, int WK,
                                         f32x4 (&acc)[MF][NF]) {
  constexpr int D = MF == 4 ? 1 : MF == 2 ? 2 : 3;
  constexpr int J = G / 32;
  const int lane = threadIdx.x & 63;
  const uint32_t lda = 2u * (uint32_t)P.k, ldw = (uint32_t)P.k / 2;
  const int groups = P.k / G;
  const Rsrc ra = rsrc_of(it.a, (uint32_t)it.rows * lda);
  Rsrc rw[NF];
  const int rows_w = (GATED ? 2 : 1) * P.n;
  const bool zeros = P.w_zeros != nullptr;
#pragma unroll
  for (int f = 0; f < NF; ++f)
    rw[f] = rsrc_of(P.w + ((uint64_t)it.e * rows_w + strip_row<NF, GATED>(P, it.strip, f)) * ldw,
                    (uint32_t)strip_rows<NF, GATED>(P, it, f) * ldw);
  const uint32_t r = lane & 15, g = lane >> 4;
  // Lane quarter q loads strip q's scales and zero points.
  const int srow = strip_row<NF, GATED>(P, it.strip, (int)g % NF) + (int)r;
  const uint64_t sat = ((uint64_t)it.e * rows_w + (srow < rows_w ? srow : rows_w - 1)) * groups;
  const uint16_t* s_p = static_cast<const uint16_t*>(P.w_scales) + sat;
  const uint8_t* z_p = P.w_zeros + sat;
  uint32_t wb[D][NF][J], sb[D], zb[D];
  v4u ab[D][MF][J];
  auto load = [&](int s, int c) {
    const bool in = c < groups;
    const uint32_t woff = in ? r * ldw + (uint32_t)c * (G / 2) + g * (G / 8) : kOutside;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      if constexpr (J == 4) {
        const v4u v = load16(rw[f], woff);
        wb[s][f][0] = v.x; wb[s][f][1] = v.y; wb[s][f][2] = v.z; wb[s][f][3] = v.w;
      } else if constexpr (J == 2) {
        const v2u v = __builtin_amdgcn_raw_buffer_load_b64(rw[f], (int)woff, 0, 0);
        wb[s][f][0] = v.x; wb[s][f][1] = v.y;
      } else {
        wb[s][f][0] = __builtin_amdgcn_raw_buffer_load_b32(rw[f], (int)woff, 0, 0);
      }
    }
    const uint32_t aoff = in ? r * lda + (uint32_t)c * (2 * G) + g * (G / 2) : kOutside;
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int j = 0; j < J; ++j)
        ab[s][m][j] = load16(ra, in ? aoff + m * 16u * lda + 16u * j : kOutside);
    const int at = in ? c : groups - 1;  // a group behind k is zeros: any scale does
    sb[s] = s_p[at];
    zb[s] = zeros ? z_p[at] : 8u;
  };
  const v4u one = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const bf16x8 ones = __builtin_bit_cast(bf16x8, one);
#pragma unroll
  for (int s = 0; s < D; ++s) load(s, kw + s * WK);
  for (int c = kw; c < groups; c += D * WK) {
#pragma unroll
    for (int s = 0; s < D; ++s) {
      const f32x4 zero = {0, 0, 0, 0};
      bf16x8 x[MF][J];
      f32x4 sum[MF];
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        sum[m] = zero;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          x[m][j] = a_like_codes(ab[s][m][j]);
          sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[m][j], ones, sum[m], 0, 0, 0);
        }
      }
      const float scale = __uint_as_float(sb[s] << 16), zero_at = 16.0f + (float)zb[s];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        f32x4 p[MF];
#pragma unroll
        for (int m = 0; m < MF; ++m) p[m] = zero;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const bf16x8 wf = codes_bf16(wb[s][f][j]);
#pragma unroll
          for (int m = 0; m < MF; ++m)
            p[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[m][j], wf, p[m], 0, 0, 0);
        }
        const bool in = c + s * WK < groups;  // else 0 * a scale that may be NaN
        const float sc = in ? __shfl(scale, f * 16 + (int)r, 64) : 0.0f;
        const float off = __shfl(zero_at, f * 16 + (int)r, 64);
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
          for (int r2 = 0; r2 < 4; ++r2)
            acc[m][f][r2] = __builtin_fmaf(sc, __builtin_fmaf(-off, sum[m][r2], p[m][r2]), acc[m][f][r2]);
      }
      load(s, c + (s + D) * WK);
    }
  }
}

// What the wavefronts of a workgroup do with items: WN lists of strips beside
// each other, k split WK ways; or (WK = 0) each wavefront alone with its own.
// Sums first, then, 16 rows at a time, the partial sums meet in LDS and the
// outputs go out, four columns a thread.
template <int WEIGHT, int G, int MF, int NF, bool GATED, bool OUT_FP8, int WN, int WK>
__device__ __forceinline__ void do_item(const GemmParams& P, const Item& it, float* part) {
  constexpr bool ALONE = WK == 0;
  constexpr int PARTS = ALONE ? 1 : WK;
  constexpr int SF = GATED ? NF / 2 : NF;   // output strips a wavefront
  constexpr int LD = NF * 16 + 4;           // floats of a partial row
  constexpr int COLS = WN * SF * 16;
  constexpr int THREADS = ALONE ? 64 : WN * WK * 64;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tid = ALONE ? lane : threadIdx.x;
  const int wn = ALONE ? 0 : wave % WN, kw = ALONE ? 0 : wave / WN;
  Item mine = it;
  mine.strip = it.strip + wn * SF;
  mine.strips = it.strips - wn * SF;
  f32x4 acc[MF][NF];
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[m][f] = f32x4{0, 0, 0, 0};
  if constexpr (WEIGHT == kWeightBf16)
    sum_bf16<MF, NF, GATED>(P, mine, kw, PARTS, acc);
  else if constexpr (WEIGHT == kWeightFp8)
    sum_fp8<MF, NF, GATED>(P, mine, kw, PARTS, acc);
  else
    sum_int4<MF, NF, GATED, G>(P, mine, kw, PARTS, acc);

  auto meet = [] {
    if constexpr (ALONE) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    } else {
      __syncthreads();
    }
  };
  const int lo = lane & 15, hi = lane >> 4;
  float* mp = part + wave * 16 * kPartLd;
  const float* first = ALONE ? mp : part;
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    if (m * 16 >= it.rows) break;  // the same for all who meet
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      if constexpr (WEIGHT == kWeightFp8) {
        *reinterpret_cast<f32x4*>(mp + lo * LD + f * 16 + 4 * hi) = acc[m][f];
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) mp[(4 * hi + r) * LD + f * 16 + lo] = acc[m][f][r];
      }
    }
    meet();
    for (int i = tid; i < 16 * COLS / 4; i += THREADS) {
      const int row = i / (COLS / 4), c4 = 4 * (i % (COLS / 4));
      const int list = c4 / (SF * 16), at = c4 % (SF * 16);
      f32x4 v = {0, 0, 0, 0}, u = {0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < PARTS; ++q) {
        const float* p = first + (q * WN + list) * 16 * kPartLd + row * LD + at;
        v += *reinterpret_cast<const f32x4*>(p);
        if constexpr (GATED) u += *reinterpret_cast<const f32x4*>(p + SF * 16);
      }
      if constexpr (GATED) {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = silu_mul(v[r], u[r]);
      }
      const int col = it.strip * 16 + c4;
      const bool in = m * 16 + row < it.rows && col < P.n && c4 < it.strips * 16;
      const uint64_t orow = (uint64_t)(it.row0 + m * 16 + row);
      if constexpr (OUT_FP8) {
        // 32 lanes hold a row's 128 columns
        float amax = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) amax = fmaxf(amax, fabsf(v[r]));  // NaN is ignored
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) amax = fmaxf(amax, __shfl_xor(amax, d, 64));
        const float inv = amax > 0.0f ? 448.0f / amax : 0.0f;
        if (in) {
          *reinterpret_cast<uint32_t*>(P.out + orow * P.n + col) =
              e4m3_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
          if (c4 == 0) P.out_scales[orow * (P.n / 128) + col / 128] = amax > 0.0f ? amax / 448.0f : 0.0f;
        }
      } else if (in) {
        *reinterpret_cast<uint2*>(P.out + 2 * (orow * P.n + col)) =
            make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
      }
    }
    meet();
  }
}

template <int WEIGHT, int G, int NF, bool GATED, bool OUT_FP8, int WN, int WK>
__device__ __forceinline__ void do_item_rows(const GemmParams& P, const Item& it, float* part) {
  if (it.rows <= 16) {
    do_item<WEIGHT, G, 1, NF, GATED, OUT_FP8, WN, WK>(P, it, part);
  } else if (it.rows <= 32) {
    do_item<WEIGHT, G, 2, NF, GATED, OUT_FP8, WN, WK>(P, it, part);
  } else if constexpr (WEIGHT == kWeightInt4 && NF == 4) {
    // registers hold 64 rows of A beside two strips
    constexpr int SF = GATED ? 1 : 2;
    Item half = it;
    half.strips = it.strips < SF ? it.strips : SF;
    do_item<WEIGHT, G, 4, NF / 2, GATED, OUT_FP8, WN, WK>(P, half, part);
    half.strip += SF;
    half.strips = it.strips - SF;
    if (half.strips > 0) do_item<WEIGHT, G, 4, NF / 2, GATED, OUT_FP8, WN, WK>(P, half, part);
  } else {
    do_item<WEIGHT, G, 4, NF, GATED, OUT_FP8, WN, WK>(P, it, part);
  }
}

// The units [u0, u1) of a list of `tiles` x `units`. A unit is an output
// strip, or (fp8 out, where a row's 128 columns share a scale) 128 columns.
template <int WEIGHT, int G, bool GATED, bool OUT_FP8, int WN, int WK>
__device__ __forceinline__ void do_run(const GemmParams& P, const uint32_t* pre, float* part, int units,
                                       uint64_t u0, uint64_t u1) {
  constexpr int SF = GATED ? kFewFrags / 2 : kFewFrags;
  if (u0 >= u1) return;
  // division in 32 bits wherever the list allows it
  uint32_t tile = u1 >> 32 ? (uint32_t)(u0 / (uint32_t)units) : (uint32_t)u0 / (uint32_t)units;
  int unit = (int)(u0 - (uint64_t)tile * units);
  int e = __builtin_amdgcn_readfirstlane(expert_of_tile(pre, P.num_experts, tile));
  uint32_t end = (uint32_t)__builtin_amdgcn_readfirstlane((int)pre[e + 1]);
  for (uint64_t left = u1 - u0; left > 0;) {
    if (unit == units) {
      unit = 0;
      if (++tile == end) {
        e = __builtin_amdgcn_readfirstlane(expert_of_tile(pre, P.num_experts, tile));
        end = (uint32_t)__builtin_amdgcn_readfirstlane((int)pre[e + 1]);
      }
    }
    const int t = (int)(tile - (uint32_t)__builtin_amdgcn_readfirstlane((int)pre[e]));
    const int c = __builtin_amdgcn_readfirstlane((int)pre[P.num_experts + 1 + e]);
    Item it;
    it.e = e;
    it.row0 = (int64_t)e * P.max_tokens + (int64_t)t * kFewRows;
    it.rows = c - t * kFewRows < kFewRows ? c - t * kFewRows : kFewRows;
    it.a = P.a + (uint64_t)it.row0 * P.k * (WEIGHT == kWeightFp8 ? 1 : 2);
    it.a_scales = WEIGHT == kWeightFp8 ? P.a_scales + (uint64_t)it.row0 * (P.k / 128) : nullptr;
    int here = units - unit;
    here = left < (uint64_t)here ? (int)left : here;
    int done = 1;
    if constexpr (OUT_FP8) {
      static_assert(WN * SF == 8, "a workgroup holds 128 columns");
      it.strip = unit * 8;
      it.strips = 8;
      do_item_rows<WEIGHT, G, kFewFrags, GATED, OUT_FP8, WN, WK>(P, it, part);
    } else if (here >= SF) {
      it.strip = unit;
      it.strips = done = SF;
      do_item_rows<WEIGHT, G, kFewFrags, GATED, OUT_FP8, WN, WK>(P, it, part);
    } else {
      // the run's last strips, fewer than a wavefront holds
      it.strip = unit;
      it.strips = 1;
      do_item_rows<WEIGHT, G, GATED ? 2 : 1, GATED, OUT_FP8, WN, WK>(P, it, part);
    }
    unit += done;
    left -= done;
  }
}

// Workgroups: two a CU (one of twice the size for the fp8 output). A power of
// two, so that the runs need no division.
constexpr int few_blocks_log2(bool out_fp8) { return out_fp8 ? 8 : 9; }

template <int WEIGHT, int G, bool GATED, bool OUT_FP8, int WN, int WK>
__global__ void __launch_bounds__(WN* WK * 64, 2) gemm_few_kernel(const GemmParams P, int most) {
  extern __shared__ __align__(16) uint8_t lds_raw[];
  __shared__ uint32_t scan[WN * WK];
  __shared__ __align__(16) float part[WN * WK * 16 * kPartLd];
  uint32_t* pre = reinterpret_cast<uint32_t*>(lds_raw);
  tile_prefix<WN * WK * 64>(P, kFewRows, 0, most, pre, scan);
  const uint32_t tiles = (uint32_t)__builtin_amdgcn_readfirstlane((int)pre[P.num_experts]);
  const int units = OUT_FP8 ? P.n / 128 : (P.n + 15) / 16;
  const uint64_t total = (uint64_t)tiles * units;
  constexpr int LOG = few_blocks_log2(OUT_FP8);
  if constexpr (!OUT_FP8) {
    // Alone a wavefront needs some strips to be busy with.
    constexpr int LOG1 = LOG + 2;
    static_assert(WN * WK == 4, "wavefronts of a workgroup");
    if (total >> LOG1 >= 2 * (GATED ? kFewFrags / 2 : kFewFrags)) {
      const uint32_t w = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      do_run<WEIGHT, G, GATED, OUT_FP8, 1, 0>(P, pre, part, units, total * w >> LOG1,
                                              total * (w + 1) >> LOG1);
      return;
    }
  }
  do_run<WEIGHT, G, GATED, OUT_FP8, WN, WK>(P, pre, part, units, total * blockIdx.x >> LOG,
                                            total * (blockIdx.x + 1) >> LOG);
}

template <int WEIGHT, int G, bool GATED, bool OUT_FP8>
hipError_t launch(const GemmParams& p, int most, hipStream_t stream) {
  constexpr int WN = OUT_FP8 ? 4 : 1, WK = OUT_FP8 ? 2 : 4;
  gemm_few_kernel<WEIGHT, G, GATED, OUT_FP8, WN, WK>
      <<<1 << few_blocks_log2(OUT_FP8), WN * WK * 64, tile_prefix_bytes(p.num_experts), stream>>>(p, most);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_few(const GemmParams& p, int most, hipStream_t stream) {
  if (p.weight == kWeightFp8) {
    if (p.out_fp8) return launch<kWeightFp8, 128, true, true>(p, most, stream);
    return p.gated ? launch<kWeightFp8, 128, true, false>(p, most, stream)
                   : launch<kWeightFp8, 128, false, false>(p, most, stream);
  }
  if (p.weight == kWeightInt4) {
    if (p.group == 128)
      return p.gated ? launch<kWeightInt4, 128, true, false>(p, most, stream)
                     : launch<kWeightInt4, 128, false, false>(p, most, stream);
    if (p.group == 64)
      return p.gated ? launch<kWeightInt4, 64, true, false>(p, most, stream)
                     : launch<kWeightInt4, 64, false, false>(p, most, stream);
    return p.gated ? launch<kWeightInt4, 32, true, false>(p, most, stream)
                   : launch<kWeightInt4, 32, false, false>(p, most, stream);
  }
  return p.gated ? launch<kWeightBf16, 128, true, false>(p, most, stream)
                 : launch<kWeightBf16, 128, false, false>(p, most, stream);
}

}  // namespace llmoe
