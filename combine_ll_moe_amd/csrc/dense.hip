// Dense products in e4m3 with a scale per 128 activations and per 128 x 128
// weights: every row through one weight.
//
// Mathematics: P[r, i] = sum over blocks b of 128 columns of
// a_scale[r, b] w_scale[i / 128, b] sum_c a[r, c] w[i, c]. Codes become bf16,
// which holds them exactly, and go through bf16 products: the matrix cores'
// own fp8 products keep a sum to about 6e-6 of its magnitudes only. A block's
// sum is scaled and added up in fp32.
//
// Design: a workgroup's wavefronts take a tile of rows by weight rows; a k step is 128
// bytes of every row, copied from memory straight into LDS some steps ahead
// of the products. A row's eight 16-byte chunks are permuted by the row's low
// bits, so that the 16 lanes that read one chunk of 16 rows meet no bank twice.
// Rows behind m or n and steps behind k are outside the buffer descriptors:
// zeros.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dense.h"
#include "expert_gemm.h"
#include "kernels.h"

namespace llmoe {
namespace {

typedef __attribute__((address_space(3))) uint8_t LdsByte;

enum : int { kPartial = 0, kPlain = 1, kGated = 2, kGatedFp8 = 3 };
constexpr int kStep = 128;  // bytes and columns of a k step

// s_waitcnt vmcnt(n) alone.
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
}

// What workgroup b of `total` does: the XCDs, to which workgroups are dealt
// in turn, take runs of the tiles, in which neighbours share rows or weights.
__device__ __forceinline__ uint32_t run_of_xcd(uint32_t b, uint32_t total) {
  const uint32_t x = b % kXcds, whole = total / kXcds, more = total % kXcds;
  return x * whole + (x < more ? x : more) + b / kXcds;
}

// WM x WN wavefronts, each FM x FN fragments of 16 x 16.
template <int WM, int WN, int FM, int FN, int STAGES, int MODE>
__global__ void __launch_bounds__(WM* WN * 64) dense_kernel(const DenseParams P, int splits) {
  constexpr int BM = WM * FM * 16, BN = WN * FN * 16, WAVES = WM * WN;
  constexpr bool GATED = MODE == kGated || MODE == kGatedFp8;
  constexpr int COLS = GATED ? BN / 2 : BN;  // output columns of a tile
  constexpr int AI = BM / 8, WI = BN / 8;    // copies of 8 rows
  constexpr int STAGE = (BM + BN) * kStep;
  static_assert(STAGES == 2 || STAGES == 4);
  static_assert(WI % WAVES == 0 && (!GATED || WI / 2 % WAVES == 0));
  static_assert(FN * 16 <= 128 && (MODE != kGatedFp8 || BN == 256));
  __shared__ __align__(16) uint8_t st0[STAGE], st1[STAGE];
  __shared__ __align__(16) uint8_t st2[STAGES > 2 ? STAGE : 16], st3[STAGES > 2 ? STAGE : 16];
  const int tid = threadIdx.x, lane = tid & 63, lo = lane & 15, hi = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int rows_w = GATED || (MODE == kPartial && P.gated) ? 2 * P.n : P.n;
  const int width = GATED ? P.n : rows_w;  // columns that the tiles cover
  const uint32_t ld = (uint32_t)P.k;
  const int kb = P.k / 128;

  const uint32_t across = (uint32_t)((width + COLS - 1) / COLS), down = (uint32_t)(((int64_t)P.m + BM - 1) / BM);
  const uint32_t tile = run_of_xcd(blockIdx.x, gridDim.x);
  const uint32_t split = tile / (across * down), at = tile % (across * down);
  // four tile columns at a time, all row tiles of those
  const uint32_t group = at / (4 * down), wide = across - 4 * group < 4 ? across - 4 * group : 4;
  const uint32_t in_g = at - 4 * down * group;
  const int64_t row0 = (int64_t)(in_g / wide) * BM;
  const int col0 = (int)((4 * group + in_g % wide) * COLS);
  const int rows = P.m - row0 < BM ? (int)(P.m - row0) : BM;
  const int cols = width - col0 < COLS ? width - col0 : COLS;
  const int k0 = (int)((int64_t)kb * split / splits), k1 = (int)((int64_t)kb * (split + 1) / splits);

  const Rsrc ra = rsrc_of(P.a + (uint64_t)row0 * ld, (uint32_t)rows * ld);
  const Rsrc rw = rsrc_of(P.w + (uint64_t)col0 * ld, (uint32_t)cols * ld);
  const Rsrc ru = rsrc_of(P.w + (uint64_t)(GATED ? P.n + col0 : 0) * ld, GATED ? (uint32_t)cols * ld : 0u);
  const uint32_t sub = (uint32_t)lane >> 3, chunk = (uint32_t)((lane & 7) ^ sub) * 16;
  auto copy = [&](int step, uint8_t* lds) __attribute__((always_inline)) {
    const uint32_t from = (uint32_t)step * kStep + chunk;
    const bool in = step < k1;
#pragma unroll
    for (int i = 0; i < (AI + WAVES - 1) / WAVES; ++i) {
      const int g = i * WAVES + wave;
      if (AI % WAVES == 0 || g < AI)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LdsByte*)(lds + g * 8 * kStep), 16,
                                                 in ? (int)((g * 8 + sub) * ld + from) : (int)kOutside, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < WI / WAVES; ++i) {
      const bool up = GATED && i >= WI / 2 / WAVES;
      const int g = i * WAVES + wave, r = up ? g - WI / 2 : g;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(up ? ru : rw, (LdsByte*)(lds + (BM + g * 8) * kStep), 16,
                                               in ? (int)((r * 8 + sub) * ld + from) : (int)kOutside, 0, 0, 0);
    }
  };

  // scales of a step: this lane's rows, and the weight blocks of this
  // wavefront's fragments. Its plain columns lie in one block; gated, its gate
  // columns do, and its up rows, which start at any multiple of 16, lie in the
  // next one from fragment `edge` on.
  const Rsrc ras = rsrc_of(P.a_scales + (uint64_t)row0 * kb, (uint32_t)rows * kb * 4u);
  const int first = GATED ? col0 + wn * (FN * 8) : col0 + wn * (FN * 16);
  const int first_up = P.n + col0 + wn * (FN * 8);
  const int last = (rows_w + 127) / 128 - 1;
  const int b0 = first / 128 < last ? first / 128 : last;
  const int b1 = first_up / 128 < last ? first_up / 128 : last, b2 = b1 < last ? b1 + 1 : last;
  const int edge = ((first_up / 128 + 1) * 128 - first_up) / 16;
  float as[2][FM], ws[2][3];
  auto scales = [&](int step, float (&av)[FM], float (&wv)[3]) __attribute__((always_inline)) {
    const int s = step < kb ? step : kb - 1;
#pragma unroll
    for (int f = 0; f < FM; ++f)
      av[f] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          ras, (int)(4u * ((uint32_t)(wm * FM * 16 + f * 16 + lo) * kb + s)), 0, 0));
    wv[0] = P.w_scales[(int64_t)b0 * kb + s];
    if constexpr (GATED) {
      wv[1] = P.w_scales[(int64_t)b1 * kb + s];
      wv[2] = P.w_scales[(int64_t)b2 * kb + s];
    }
  };

  // LDS row of weight fragment f: gated, fragments from FN / 2 on are the up
  // rows of the same columns.
  auto frag_row = [&](int f) {
    if constexpr (GATED)
      return (f < FN / 2 ? 0 : BN / 2) + wn * (FN * 8) + (f % (FN / 2)) * 16;
    else
      return wn * FN * 16 + f * 16;
  };
  auto chunk_of = [&](const uint8_t* lds, int r, int c) {
    return *reinterpret_cast<const v4u*>(lds + r * kStep + ((c ^ (r & 7)) << 4));
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int f = 0; f < FN; ++f) acc[m][f] = f32x4{0, 0, 0, 0};
  auto multiply = [&](const uint8_t* lds, const float (&av)[FM], const float (&wv)[3]) __attribute__((always_inline)) {
    Bf16x16 a[FM][2];
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j) a[m][j] = fp8_to_bf16(chunk_of(lds, wm * FM * 16 + m * 16 + lo, 4 * j + hi));
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      Bf16x16 w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) w[j] = fp8_to_bf16(chunk_of(lds + BM * kStep, frag_row(f) + lo, 4 * j + hi));
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        f32x4 p = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j].lo, a[m][j].lo, p, 0, 0, 0);
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j].hi, a[m][j].hi, p, 0, 0, 0);
        }
        const float sc = av[m] * wv[!GATED || f < FN / 2 ? 0 : f - FN / 2 < edge ? 1 : 2];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[m][f][r] = __builtin_fmaf(sc, p[r], acc[m][f][r]);
      }
    }
  };

  // A step's copies are waited for, then all wavefronts meet: the step is
  // whole, and the buffer of the one before it free for the copies of the
  // step STAGES - 1 ahead. Only the copies of the steps between may be under way.
  constexpr int AHEAD = STAGES - 1;
  uint8_t* const buffers[4] = {st0, st1, st2, st3};
#pragma unroll
  for (int s = 0; s < AHEAD; ++s) copy(k0 + s, buffers[s]);
  scales(k0, as[0], ws[0]);
  for (int k = k0; k < k1; k += STAGES) {
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      if (k + s < k1) {
        wait_loads<0>();
        __syncthreads();
        copy(k + s + AHEAD, buffers[(s + AHEAD) % STAGES]);
        scales(k + s + 1, as[(s + 1) & 1], ws[(s + 1) & 1]);
        multiply(buffers[s], as[s & 1], ws[s & 1]);
      }
    }
  }

  constexpr int F = GATED ? FN / 2 : FN;
  if constexpr (GATED) {
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[m][f][q] = silu_mul(acc[m][f][q], acc[m][f + F][q]);
  }
  float* amaxes = reinterpret_cast<float*>(st0);  // fp8: amax of a row's part, [BM][WN]
  if constexpr (MODE == kGatedFp8) {
    wait_loads<0>();
    __syncthreads();  // copies behind the last step have landed
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      float v = 0.0f;
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) v = fmaxf(v, fabsf(acc[m][f][q]));  // NaN is ignored
      v = fmaxf(v, __shfl_xor(v, 16, 64));
      v = fmaxf(v, __shfl_xor(v, 32, 64));
      if (hi == 0) amaxes[(wm * FM * 16 + m * 16 + lo) * WN + wn] = v;
    }
    __syncthreads();
  }
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const int row = wm * FM * 16 + m * 16 + lo;
    if (row >= rows) continue;
    const uint64_t orow = (uint64_t)(row0 + row);
    float inv = 0.0f;
    if constexpr (MODE == kGatedFp8) {
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < WN; ++i) amax = fmaxf(amax, amaxes[row * WN + i]);
      const BlockScale s = block_scale(amax);
      inv = s.inv;
      if (wn == 0 && hi == 0) P.out_scales[orow * (P.n / 128) + col0 / 128] = s.scale;
    }
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int col = wn * F * 16 + f * 16 + 4 * hi;
      if (col >= cols) continue;
      f32x4 v = acc[m][f];
      const uint64_t to = orow * width + col0 + col;
      if constexpr (MODE == kPartial) {
        *reinterpret_cast<f32x4*>(P.partial + (uint64_t)split * P.m * width + to) = v;
      } else if constexpr (MODE == kGatedFp8) {
        *reinterpret_cast<uint32_t*>(P.out + to) = e4m3_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
      } else {
        if (MODE == kPlain && P.addend) v += *reinterpret_cast<const f32x4*>(P.addend + to);
        if (MODE == kPlain && P.out_type == kOutFp32)
          *reinterpret_cast<f32x4*>(P.out + 4 * to) = v;
        else
          *reinterpret_cast<uint2*>(P.out + 2 * to) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
      }
    }
  }
}

// The product of `rows` rows from row `first` on.
DenseParams rows_from(const DenseParams& p, uint64_t first, int rows) {
  DenseParams q = p;
  q.a += first * p.k;
  q.a_scales += first * (p.k / 128);
  if (q.addend) q.addend += first * p.n;
  q.out += first * p.n * (p.out_type == kOutFp8 ? 1 : p.out_type == kOutFp32 ? 4 : 2);
  if (p.out_type == kOutFp8) q.out_scales += first * (p.n / 128);
  q.m = rows;
  return q;
}

template <int WM, int WN, int FM, int FN, int STAGES, int MODE>
hipError_t launch(const DenseParams& p, hipStream_t stream) {
  constexpr int BM = WM * FM * 16, BN = WN * FN * 16, THREADS = WM * WN * 64;
  constexpr int COLS = MODE == kGated || MODE == kGatedFp8 ? BN / 2 : BN;
  // a grid has fewer than 2^32 threads: more rows go out in several launches
  const int64_t across = ((int64_t)p.n + COLS - 1) / COLS;
  const int64_t most = ((1ll << 31) / THREADS / across) * BM;
  for (int64_t first = 0; first < p.m; first += most) {
    const DenseParams q = rows_from(p, (uint64_t)first, (int)(p.m - first < most ? p.m - first : most));
    const int64_t tiles = across * (((int64_t)q.m + BM - 1) / BM);
    dense_kernel<WM, WN, FM, FN, STAGES, MODE><<<(unsigned)tiles, THREADS, 0, stream>>>(q, 1);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_dense(const DenseParams& p, hipStream_t stream) {
  if (p.m == 0) return hipSuccess;
  if (!p.gated) return launch<1, 4, 4, 4, 2, kPlain>(p, stream);
  return p.out_type == kOutFp8 ? launch<1, 4, 4, 4, 2, kGatedFp8>(p, stream)
                               : launch<1, 4, 4, 4, 2, kGated>(p, stream);
}

}  // namespace llmoe
