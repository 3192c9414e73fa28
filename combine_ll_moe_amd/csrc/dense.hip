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
// of the products, the scales with it. A row's eight 16-byte chunks are
// permuted by the row's low bits, so that the 16 lanes that read one chunk of
// 16 rows meet no bank twice. Rows behind m or n and steps behind k are outside
// the buffer descriptors: zeros. Where tiles alone do not fill the GPU, runs of
// k go to workgroups of their own, whose sums meet in the workspace and are
// finished by a second kernel; few rows have a kernel that needs no second one
// (launch_dense says which sizes take which).
//
// Bound: few rows are latency and a second launch (one row, gated, n 2048, k
// 7168, 29 MB: 8.3 us to bf16, 10.8 to fp8, of which 2.0 are the second
// kernel and the rest its launch). Many rows: 8192 x 4096 x 7168 take 400 us, 1.2 PFLOP/s; the copies
// alone take 203 of them and the products without copies 340, which overlap no
// better: a SIMD's matrix unit is busy 50 % of the time, and 2.8 vector
// instructions a product (conversion and scaling) share its wavefronts' issue.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dense.h"
#include "layout.h"
#include "ll_moe.h"
#include "tile.h"

namespace llmoe {
namespace {

enum : int { kPartial = 0, kPlain = 1, kGated = 2, kGatedFp8 = 3 };
static_assert(kStep == kFp8Block);  // a k step is one scale's columns
constexpr int64_t kWorkspace = LL_MOE_DENSE_WORKSPACE;
// Few steps of k; CUs; up to so many tiles there are 64 x 64 ones, with many
// steps and with few; rows up to which a tile has 16, 64 and 128 of them all the
// same; steps of k that a split has to save, to be worth its second kernel (1 row,
// n 7168, k 2048: 7.2 us, in two runs 8.2).
constexpr int kShort = 40, kShortGated = 24;
constexpr int64_t kCus = 256;
constexpr int kTiles64 = 512, kTiles64Deep = 256, kTiles64Gated = 256, kTiles64GatedDeep = 128;
constexpr int kTokens16 = 32, kTokens16Gated = 16, kTokens64 = 64, kTokens128 = 4096;
constexpr int kWorthSplit = 12;

// WM x WN wavefronts, each FM x FN fragments of 16 x 16; STAGES buffers of a
// step in LDS. The steps of k are divided among `splits` workgroups.
template <int WM, int WN, int FM, int FN, int STAGES, int MODE>
__global__ void __launch_bounds__(WM* WN * 64, 2) dense_kernel(const DenseParams P, int splits) {
  constexpr int BM = WM * FM * 16, BN = WN * FN * 16, WAVES = WM * WN;
  constexpr bool GATED = MODE == kGated || MODE == kGatedFp8;
  constexpr int COLS = GATED ? BN / 2 : BN;  // output columns of a tile
  constexpr int AI = BM / 8, WI = BN / 8;    // copies of 8 rows
  constexpr int AC = (AI + WAVES - 1) / WAVES, WC = WI / WAVES;  // of a wavefront
  constexpr int SCALES = (BM + BN) * kStep;  // in a stage: 512 bytes of scales a wavefront
  constexpr int STAGE = SCALES + WAVES * 512;
  static_assert(FM <= 4);
  static_assert(STAGES >= 2 && STAGES <= 4);
  static_assert(WI % WAVES == 0 && (AI % WAVES == 0 || WAVES % AI == 0) && (!GATED || WI / 2 % WAVES == 0));
  static_assert(FN * 16 <= 128 && (MODE != kGatedFp8 || BN == 256));
  // an array each, so that the compiler can tell a step's copies from the
  // reads of another one's
  __shared__ __align__(16) uint8_t st0[STAGE], st1[STAGE];
  __shared__ __align__(16) uint8_t st2[STAGES > 2 ? STAGE : 16], st3[STAGES > 3 ? STAGE : 16];
  const int tid = threadIdx.x, lane = tid & 63, lo = lane & 15, hi = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int rows_w = P.gated ? 2 * P.n : P.n;
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
  const uint32_t sub = (uint32_t)lane >> 3, mine = sub * ld + ((lane & 7) ^ sub) * 16;
  // Scales of a step: of this wavefront's rows, a lane each, and of the weight
  // blocks of its fragments, in lanes 0 to 2. Its plain columns lie in one
  // block; gated, its gate columns do, and its up rows, which start at any
  // multiple of 16, lie in the next one from fragment `edge` on.
  const Rsrc ras = rsrc_of(P.a_scales + (uint64_t)row0 * kb, (uint32_t)rows * kb * 4u);
  const int last = (rows_w + 127) / 128 - 1;
  const int first = GATED ? col0 + wn * (FN * 8) : col0 + wn * (FN * 16);
  const int first_up = P.n + first;
  const int edge = ((first_up / 128 + 1) * 128 - first_up) / 16;
  const int block = !GATED || lane == 0 ? first / 128 : first_up / 128 + (lane > 1);
  const Rsrc rws = rsrc_of(P.w_scales, (uint32_t)(last + 1) * kb * 4u);
  const uint32_t my_row = 4u * (uint32_t)((wm * FM * 16 + (lane & (FM * 16 - 1))) * kb);
  const uint32_t my_block = 4u * (uint32_t)((block < last ? block : last) * kb);

  // Everything of a step: the copies into its buffer, and its scales. Every
  // wavefront issues the same number of loads, steps behind k1 too (those read
  // nothing): the waits count them.
  constexpr int LOADS = AC + WC + 2;
  auto fetch = [&](int step, uint8_t* lds) __attribute__((always_inline)) {
    // offsets: the lane's own and a uniform part, which is outside every
    // descriptor behind k1
    const uint32_t at = step < k1 ? (uint32_t)step * kStep : kOutside;
#pragma unroll
    for (int i = 0; i < AC; ++i) {
      const int g = AI < WAVES ? wave % AI : i * WAVES + wave;
      copy16(ra, lds + g * 8 * kStep, mine + (g * 8 * ld + at));
    }
#pragma unroll
    for (int i = 0; i < WC; ++i) {
      const bool up = GATED && i >= WC / 2;
      const int g = i * WAVES + wave, r = up ? g - WI / 2 : g;
      copy16(up ? ru : rw, lds + (BM + g * 8) * kStep, mine + (r * 8 * ld + at));
    }
    const uint32_t s = step < k1 ? 4u * (uint32_t)step : kOutside;
    uint8_t* scales = lds + SCALES + wave * 512;
    copy4(ras, scales, my_row + s);
    copy4(rws, scales + 256, my_block + s);
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
  auto multiply = [&](const uint8_t* lds) __attribute__((always_inline)) {
    const float* scales = reinterpret_cast<const float*>(lds + SCALES + wave * 512);
    float av[FM];
#pragma unroll
    for (int m = 0; m < FM; ++m) av[m] = scales[m * 16 + lo];
    const float w0 = scales[64], w1 = GATED ? scales[65] : 0.0f, w2 = GATED ? scales[66] : 0.0f;
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
        const float sc = av[m] * (!GATED || f < FN / 2 ? w0 : f - FN / 2 < edge ? w1 : w2);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[m][f][r] = __builtin_fmaf(sc, p[r], acc[m][f][r]);
      }
    }
  };

  // A step's loads are waited for, those of the steps behind it still under
  // way, then all wavefronts meet: the step is whole, and the buffer of the one
  // before it is free for the step STAGES - 1 ahead.
  constexpr int AHEAD = STAGES - 1;
  uint8_t* const buffers[4] = {st0, st1, st2, st3};
#pragma unroll
  for (int s = 0; s < AHEAD; ++s) fetch(k0 + s, buffers[s]);
  // Steps behind k1 are zeros: whole rounds of STAGES, without branches.
  for (int k = k0; k < k1; k += STAGES) {
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
    __syncthreads();  // copies behind the last step have landed, of all wavefronts
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

// A few rows: 16 or 32 rows of A by 16 of W, whose columns the wavefronts split
// and whose sums meet in LDS, so that one launch does it. Gated, the 16 are 8
// gate rows and the 8 up rows of the same columns; their values go out in bf16,
// or (kValues) in fp32 to the workspace, for dense_finish_kernel to quantize.
// Rows come by whole lines into registers, a step ahead, and through LDS into
// the products' order. Eight wavefronts, so that a CU has up to four workgroups
// under way (one row, gated to bf16, n 2048, k 7168: 8.3 us, with sixteen 9.1;
// two steps ahead 8.4).
enum : int { kValues = 4 };
template <int FM, int MODE>
__global__ void __launch_bounds__(512) dense_few_kernel(const DenseParams P) {
  constexpr bool GATED = MODE != kPlain;
  constexpr int WAVES = 8;
  constexpr int ROWS = 16 * FM, COLS = GATED ? 8 : 16, PART = 16 * kStep;
  __shared__ __align__(16) uint8_t pool[WAVES * (FM + 1) * PART];
  const int lane = threadIdx.x & 63, lo = lane & 15, hi = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t ld = (uint32_t)P.k;
  const int kb = P.k / 128;
  const int s0 = kb * wave / WAVES, s1 = kb * (wave + 1) / WAVES;
  const uint32_t across = (uint32_t)(P.n / COLS);
  const int64_t row0 = (int64_t)(blockIdx.x / across) * ROWS;
  const int col0 = (int)(blockIdx.x % across) * COLS;
  const int rows = P.m - row0 < ROWS ? (int)(P.m - row0) : ROWS;
  const int second = GATED ? P.n + col0 : col0 + 8;  // rows 8-15 of W
  const Rsrc ra = rsrc_of(P.a + (uint64_t)row0 * ld, (uint32_t)rows * ld);
  const Rsrc rw0 = rsrc_of(P.w + (uint64_t)col0 * ld, 8 * ld), rw1 = rsrc_of(P.w + (uint64_t)second * ld, 8 * ld);
  const Rsrc ras = rsrc_of(P.a_scales + (uint64_t)row0 * kb, (uint32_t)rows * kb * 4u);
  const Rsrc rws = rsrc_of(P.w_scales, (uint32_t)((GATED ? 2 * P.n : P.n) + 127) / 128 * kb * 4u);
  const uint32_t my_block = 4u * (uint32_t)((hi < 2 ? col0 : second) / 128 * kb);
  uint8_t* al = pool + wave * (FM + 1) * PART;  // rows of W, then of A
  uint32_t apart = 0;
  asm volatile("" : "+v"(apart));  // lanes read each other's rows: no read moves across the writes
  const uint8_t* ar = al + apart;
  const uint32_t r8 = (uint32_t)lane >> 3, mine = r8 * ld + (lane & 7) * 16;

  v4u ab[2 * FM], wb[2];
  float as[FM], ws;
  auto load = [&](int step) {
    const uint32_t at = step < s1 ? (uint32_t)step * kStep : kOutside, sc = step < s1 ? 4u * (uint32_t)step : kOutside;
    wb[0] = __builtin_amdgcn_raw_buffer_load_b128(rw0, (int)(mine + at), 0, 0);
    wb[1] = __builtin_amdgcn_raw_buffer_load_b128(rw1, (int)(mine + at), 0, 0);
#pragma unroll
    for (int i = 0; i < 2 * FM; ++i)
      ab[i] = __builtin_amdgcn_raw_buffer_load_b128(ra, (int)(mine + 8 * i * ld + at), 0, 0);
#pragma unroll
    for (int m = 0; m < FM; ++m)
      as[m] = __uint_as_float(
          __builtin_amdgcn_raw_buffer_load_b32(ras, (int)(4u * (uint32_t)((16 * m + lo) * kb) + sc), 0, 0));
    ws = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rws, (int)(my_block + sc), 0, 0));
  };
  auto store = [&] {
    const uint32_t at = r8 * kStep + (((lane & 7) ^ r8) & 7) * 16;
    *reinterpret_cast<v4u*>(al + at) = wb[0];
    *reinterpret_cast<v4u*>(al + 8 * kStep + at) = wb[1];
#pragma unroll
    for (int i = 0; i < 2 * FM; ++i) *reinterpret_cast<v4u*>(al + PART + 8 * i * kStep + at) = ab[i];
  };
  auto chunk = [&](int part, int c) {
    return fp8_to_bf16(*reinterpret_cast<const v4u*>(ar + part + lo * kStep + ((c ^ lo) & 7) * 16));
  };
  f32x4 acc[FM];
#pragma unroll
  for (int m = 0; m < FM; ++m) acc[m] = f32x4{0, 0, 0, 0};
  load(s0);
  for (int k = s0; k < s1; ++k) {
    store();
    float sc[FM];
#pragma unroll
    for (int m = 0; m < FM; ++m) sc[m] = as[m] * ws;
    load(k + 1);
    const Bf16x16 w[2] = {chunk(0, hi), chunk(0, 4 + hi)};
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      f32x4 p = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const Bf16x16 a = chunk((m + 1) * PART, 4 * j + hi);
        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j].lo, a.lo, p, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j].hi, a.hi, p, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[m][r] = __builtin_fmaf(sc[m], p[r], acc[m][r]);
    }
  }
  // the wavefronts' sums meet: lane l holds W rows 4 (l / 16) + r of row l % 16
  __syncthreads();
  float* sums = reinterpret_cast<float*>(pool);
#pragma unroll
  for (int m = 0; m < FM; ++m)
    *reinterpret_cast<f32x4*>(sums + wave * (ROWS * 16) + (16 * m + lo) * 16 + 4 * hi) = acc[m];
  __syncthreads();
  const int t = threadIdx.x;
  static_assert(ROWS * COLS <= WAVES * 64);
  if (t < ROWS * COLS) {
    const int r = t / COLS, c = t % COLS;
    float v = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      v += sums[w * (ROWS * 16) + r * 16 + c];
      if (GATED) u += sums[w * (ROWS * 16) + r * 16 + 8 + c];
    }
    if (GATED) v = silu_mul(v, u);
    if (r < rows) {
      const uint64_t to = (uint64_t)(row0 + r) * P.n + col0 + c;
      if (MODE == kPlain && P.addend) v += P.addend[to];
      if (MODE == kValues) P.partial[to] = v;
      else if (MODE == kPlain && P.out_type == kOutFp32) reinterpret_cast<float*>(P.out)[to] = v;
      else reinterpret_cast<uint16_t*>(P.out)[to] = (uint16_t)bf16_pair(v, 0.0f);
    }
  }
}

// The partial sums of `splits` runs of k to outputs: a thread has four columns
// of a row, 32 of them a block of 128 columns.
__global__ void __launch_bounds__(256) dense_finish_kernel(const DenseParams P, int splits) {
  const int blocks = (P.n + 127) / 128;
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = item / 32 / blocks;
  const int col = (int)(item / 32 % blocks) * 128 + (int)(item & 31) * 4;
  const int width = P.gated ? 2 * P.n : P.n;
  const bool in = row < P.m && col < P.n;
  f32x4 v = {0, 0, 0, 0}, u = {0, 0, 0, 0};
  if (in) {
    const float* at = P.partial + row * width + col;
    for (int s = 0; s < splits; ++s) {
      v += *reinterpret_cast<const f32x4*>(at);
      if (P.gated) u += *reinterpret_cast<const f32x4*>(at + P.n);
      at += (int64_t)P.m * width;
    }
  }
  if (P.gated)
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = silu_mul(v[q], u[q]);
  const uint64_t to = (uint64_t)row * P.n + col;
  if (P.out_type == kOutFp8) {
    float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));  // NaN is ignored
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) amax = fmaxf(amax, __shfl_xor(amax, d, 64));
    const BlockScale s = block_scale(amax);
    if (!in) return;
    *reinterpret_cast<uint32_t*>(P.out + to) = e4m3_pack4(v[0] * s.inv, v[1] * s.inv, v[2] * s.inv, v[3] * s.inv);
    if ((item & 31) == 0) P.out_scales[row * blocks + col / 128] = s.scale;
    return;
  }
  if (!in) return;
  if (P.addend) v += *reinterpret_cast<const f32x4*>(P.addend + to);
  if (P.out_type == kOutFp32)
    *reinterpret_cast<f32x4*>(P.out + 4 * to) = v;
  else
    *reinterpret_cast<uint2*>(P.out + 2 * to) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
}

hipError_t launch_finish(const DenseParams& p, int splits, hipStream_t stream) {
  const int64_t threads = (int64_t)p.m * ((p.n + 127) / 128) * 32;
  dense_finish_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, stream>>>(p, splits);
  return hipGetLastError();
}

template <int FM>
hipError_t launch_few(const DenseParams& p, hipStream_t stream) {
  const unsigned blocks = (unsigned)(((int64_t)p.m + 16 * FM - 1) / (16 * FM) * (p.n / (p.gated ? 8 : 16)));
  if (!p.gated) dense_few_kernel<FM, kPlain><<<blocks, 512, 0, stream>>>(p);
  else if (p.out_type == kOutFp8) dense_few_kernel<FM, kValues><<<blocks, 512, 0, stream>>>(p);
  else dense_few_kernel<FM, kGated><<<blocks, 512, 0, stream>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.out_type != kOutFp8) return e;
  DenseParams q = p;
  q.gated = 0;  // the values are already one each
  return launch_finish(q, 1, stream);
}

// Through partial sums in the workspace, which they fit.
template <int WM, int WN, int FM, int FN, int STAGES>
hipError_t launch_split(const DenseParams& p, int splits, hipStream_t stream) {
  constexpr int BM = WM * FM * 16, BN = WN * FN * 16;
  const int64_t width = p.gated ? 2 * (int64_t)p.n : p.n;
  const int64_t tiles = (width + BN - 1) / BN * (((int64_t)p.m + BM - 1) / BM) * splits;
  dense_kernel<WM, WN, FM, FN, STAGES, kPartial><<<(unsigned)tiles, WM * WN * 64, 0, stream>>>(p, splits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_finish(p, splits, stream);
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

// Which tiles, and how many runs of k, by the sizes. The figures are us of
// one call, its weights out of the caches, gated to fp8 with n 2048 and k 7168
// | plain, to fp32 with an addend, with n 7168 and k 2048, unless said otherwise.
hipError_t launch_dense(const DenseParams& p, hipStream_t stream) {
  if (p.m == 0) return hipSuccess;
  const int64_t rows_w = p.gated ? 2 * (int64_t)p.n : p.n, kb = p.k / 128;
  const int64_t bytes = (int64_t)p.m * rows_w * 4;  // of one set of partial sums
  auto tiles = [&](int64_t bm, int64_t bn) { return (rows_w + bn - 1) / bn * ((p.m + bm - 1) / bm); };
  // Runs of k for so many tiles: as many as `room` workgroups allow, of 7
  // steps or more, and `least` if there are so many steps.
  auto runs = [&](int64_t n, int64_t room, int64_t least) {
    int64_t s = room / n;
    if (s < least) s = least;
    if (s > kb / 7) s = kb / 7;
    if (s > kWorkspace / bytes) s = kWorkspace / bytes;
    return s < 1 ? 1 : s;
  };
  // 16 x 16 or 32 x 16 while those are few. To bf16, n 2048: 1 row 8.3 (16 x 64
  // tiles in two runs of k 13.5), 17 rows in 32 x 16 10.1 (16 x 16 12.3, 64 x 64
  // 14.7), 32 rows 12.8 (14.1, 15.1); 64 rows of n 1536, k 2048 in 16 x 16 6.5
  // (9.7), k 7168 16.8 (16.4); 16 rows of n 2560, k 7168 16.3 (15.0). | 1 row 5.4
  // (7.0), 16 rows 6.2 (7.4). To fp8 the second kernel is needed all the same: 1
  // row 10.8 (12.0 in four), n and k 4096 11.4 (11.0), 16 rows 13.4 (11.9), n 4096
  // and k 1024 6.5 (7.5). 64 rows of n 3584, k 2048, plain in 32 x 16 7.0 (9.7), k
  // 7168 19.0 (16.4).
  const bool fp8 = p.out_type == kOutFp8, few_steps = kb <= (fp8 ? kShortGated : kShort);
  const int64_t strips = p.n / (p.gated ? 8 : 16);
  const int64_t of16 = ((int64_t)p.m + 15) / 16 * strips, of32 = ((int64_t)p.m + 31) / 32 * strips;
  if (p.m > 16 && of16 > kCus && of32 <= kCus) return launch_few<2>(p, stream);
  const bool less = p.gated && !few_steps && (fp8 || (p.m > 8 && p.m <= 16));
  if (of16 <= (less ? kCus : 3 * kCus)) return launch_few<1>(p, stream);
  if (p.m > 16 && of32 <= 2 * kCus && few_steps) return launch_few<2>(p, stream);
  // 16 x 64: 16 rows, gated, n 4096, k 7168 16.1 in two runs (16 x 16 19.1, 64 x
  // 64 20.0); plain, n 16384, k 2048 8.5 (11.1, 10.6)
  if (p.gated && p.m <= kTokens16Gated && bytes <= kWorkspace)
    return launch_split<1, 4, 1, 1, 4>(p, (int)runs(tiles(16, 64), 256, 2), stream);
  if (!p.gated && p.m <= kTokens16) return launch<1, 4, 1, 1, 4, kPlain>(p, stream);
  // 64 x 64: 64 rows 16.8 (16 x 64 24.1), 128 rows 21.9 (128 x 128 23.9) | 11.3
  // and 11.9 (128 x 128 15.6 in two runs), 256 rows 32 (29) | 18.2 (23.5). To
  // bf16, plain, n 2048: 512 rows, k 2048 10.7 (128 x 128 19.1), k 7168 30.4
  // (29.5); 1024 rows, k 2048 17.3 (21.4), k 7168 50.4 (43.8). Gated, n 1024: 256
  // rows, k 1024 9.5 (13.2), k 7168 21.5 (26.3); 512 rows, k 1024 11.3 (15.4), k
  // 7168 31.8 (30.0)
  const int64_t most64 = p.gated ? (kb > kShortGated ? kTiles64GatedDeep : kTiles64Gated)
                                 : (few_steps ? kTiles64 : kTiles64Deep);
  if (p.m <= kTokens64 || tiles(64, 64) <= most64) {
    const int64_t s = runs(tiles(64, 64), 256, 1);
    if ((p.gated && bytes <= kWorkspace) || kb - kb / s >= kWorthSplit)
      return launch_split<2, 2, 2, 2, 4>(p, (int)s, stream);
    if (!p.gated) return launch<2, 2, 2, 2, 4, kPlain>(p, stream);
  }
  // Gated, many rows: 256 x 256, a tile a CU, as many rows as fill the CUs a
  // whole number of times (8192 rows 412, in 128 x 256 480; to bf16 400, in 128 x
  // 128 422). What is left goes by its own size, unless it nearly fills them too
  // (3300 rows 195, in 128 x 128 211) or its sums do not fit the workspace (5000
  // rows 264, all in 256 x 256 387; n 256, k 4096, 8192 rows in 128 x 128 46, 111).
  if (p.gated) {
    const int64_t across = ((int64_t)p.n + 127) / 128, fill = across < kCus ? kCus / across * 256 : 256;
    const int64_t rest = p.m % fill, whole = rest * 4 > fill * 3 || rest * rows_w * 4 > kWorkspace ? p.m : p.m - rest;
    if (whole > 0) {
      const DenseParams q = rows_from(p, 0, (int)whole);
      const hipError_t e = p.out_type == kOutFp8 ? launch<4, 2, 4, 8, 2, kGatedFp8>(q, stream)
                                                 : launch<4, 2, 4, 8, 2, kGated>(q, stream);
      if (e != hipSuccess || whole == p.m) return e;
      return launch_dense(rows_from(p, (uint64_t)whole, (int)rest), stream);
    }
  }
  // 128 x 128, two workgroups a CU: 777 rows 62 in two runs (71 in one, 128 x
  // 256 68 to 107) | 36 (128 x 256 42, 64 x 64 and less 62); 8192 rows | 239
  // (256 x 256 250)
  // Gated and deep, rows little beyond 256 or 512 of those tiles go out in two
  // parts, too (1100 rows 90, together 105; 2200 rows 143, 160).
  if (p.gated && kb > kShortGated) {
    const int64_t fill = kCus / ((rows_w + 127) / 128) * 128, rest = fill ? p.m % fill : 0, times = fill ? p.m / fill : 0;
    if (rest > 0 && ((times == 1 && rest * 4 <= fill) || (times == 2 && rest * 2 <= fill))) {
      const hipError_t e = launch_dense(rows_from(p, 0, (int)(p.m - rest)), stream);
      return e != hipSuccess ? e : launch_dense(rows_from(p, (uint64_t)(p.m - rest), (int)rest), stream);
    }
  }
  const int64_t s = runs(tiles(128, 128), 512, 1);
  if (p.gated || (p.m <= kTokens128 && kb - kb / s >= kWorthSplit))
    return launch_split<2, 2, 4, 4, 2>(p, (int)s, stream);
  return launch<2, 2, 4, 4, 2, kPlain>(p, stream);
}

}  // namespace llmoe
