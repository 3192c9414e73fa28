// Products grouped by expert, for experts with many rows: tiles of 256 rows
// and 256 weight rows on the matrix cores.
//
// Mathematics: as gemm_few.h, P = A W^T over an expert's rows. fp8 codes
// become bf16, which holds them exactly, and go through bf16 products at half
// the rate: the matrix cores keep a sum of fp8 products to about 6e-6 of the
// products' magnitudes only (measured over 128 columns, of one 128-column
// product and of four 32-column ones), a bf16 product to fp32's rounding. With
// fp8 products a bf16 output was rounded to another value than the exact
// sum's 80 times as often, and went by which kernel a row fell to.
//
// Design: eight wavefronts, 4 x 2, each 64 rows by 128 weight rows. A k step
// is 128 bytes of every row (64 bf16, 128 fp8): 64 KiB, copied from memory
// straight into LDS while the step before it is multiplied, in two buffers.
// A row's eight 16-byte chunks are permuted by the row's low bits, so that
// the 16 lanes that read one chunk of 16 rows meet no bank twice; the copy
// writes LDS in lane order, so it is the lanes' addresses that are permuted.
// Rows behind the expert's count or behind n and columns behind k are outside
// the buffer descriptors: zeros. A row quarter without rows is skipped; each
// SIMD holds wavefronts of two quarters.
//
// Bound: the copies, which land later than a step's products end. 8 experts of
// 2048 rows, 4096 weight rows x 4096 columns (calls one by one): bf16 548-554
// us (992-1004 TFLOP/s; 430 remained without any copy of one run's 612), gated
// 565-596; fp8, where the codes' conversion comes beside the products, 547-549
// (fp8 products took 412), gated 591-612 to bf16 and 588-591 to fp8; 4-bit
// weights, where the scaling of every group's sums adds vector instructions,
// 839-853 in groups of 128 (645-655 TFLOP/s), gated 894-939, and 1140-1154 in
// groups of 32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_gemm.h"
#include "kernels.h"

namespace llmoe {
namespace {

constexpr int kTile = kTileRows;      // rows of a tile, and weight rows
constexpr int kStepBytes = 128;       // of a row in a k step
constexpr int kHalf = kTile * kStepBytes;
constexpr int kThreads = 512;


typedef __attribute__((address_space(3))) uint8_t LdsByte;

// What a wavefront copies of a k step: 32 rows of A and 32 of W, 8 rows an
// instruction, lane l row l / 8 and slot l % 8 of it.
struct Source {
  Rsrc a, w;
  uint32_t a_off, w_off;  // this lane's first row and chunk
  uint32_t ld;            // row bytes
  uint32_t chunk;         // byte of this lane's chunk in a step
};

__device__ __forceinline__ void copy_step(const Source& s, int step, uint8_t* lds, int wave) {
  const uint32_t at = (uint32_t)step * kStepBytes + s.chunk;
  const bool in = at < s.ld;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t rows = (uint32_t)i * 8 * s.ld;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        s.a, (LdsByte*)(lds + (wave * 32 + i * 8) * kStepBytes), 16,
        in ? (int)(s.a_off + rows + at) : (int)kOutside, 0, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        s.w, (LdsByte*)(lds + kHalf + (wave * 32 + i * 8) * kStepBytes), 16,
        in ? (int)(s.w_off + rows + at) : (int)kOutside, 0, 0, 0);
  }
}

// 16 bytes of chunk c of row r.
__device__ __forceinline__ v4u chunk_of(const uint8_t* lds, int r, int c) {
  return *reinterpret_cast<const v4u*>(lds + r * kStepBytes + ((c ^ (r & 7)) << 4));
}

// LDS row of weight fragment f of column half wn. Gated tiles hold 128 gate
// rows, then 128 up rows; a wavefront's fragments 0-3 are gate rows, 4-7 the
// up rows of the same columns.
template <bool GATED>
__device__ __forceinline__ int frag_row(int wn, int f) {
  return GATED ? (f < 4 ? 0 : 128) + wn * 64 + (f & 3) * 16 : wn * 128 + f * 16;
}

// One k step. acc[m][f]: lane l holds weight rows 4 (l / 16) + r of fragment
// f for row l % 16 of row fragment m.
template <int WEIGHT, bool GATED>
__device__ __forceinline__ void multiply(const uint8_t* lds, int wm, int wn, const float (&as)[4],
                                         const float (&ws)[3], int edge, f32x4 (&acc)[4][8]) {
  const int lane = threadIdx.x & 63, lo = lane & 15, hi = lane >> 4;
  const uint8_t* la = lds;
  const uint8_t* lw = lds + kHalf;
  if constexpr (WEIGHT == kWeightBf16) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      v4u a[4], w[8];
#pragma unroll
      for (int m = 0; m < 4; ++m) a[m] = chunk_of(la, wm * 64 + m * 16 + lo, 4 * j + hi);
#pragma unroll
      for (int f = 0; f < 8; ++f) w[f] = chunk_of(lw, frag_row<GATED>(wn, f) + lo, 4 * j + hi);
#pragma unroll
      for (int f = 0; f < 8; ++f)
#pragma unroll
        for (int m = 0; m < 4; ++m)
          acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, w[f]), __builtin_bit_cast(bf16x8, a[m]), acc[m][f], 0, 0, 0);
    }
  } else {
    // Gated: the step's halves in turn, for the registers (8 experts of 2048
    // rows, 8192 weight rows x 4096, to bf16 1365 us against 1454, to fp8 1296
    // against 1294; plain, 4096 weight rows, where the halves' own scaling
    // costs more, 610 against 561).
    constexpr int HALVES = GATED ? 2 : 1, CHUNKS = 2 / HALVES;
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      Bf16x16 a[4][CHUNKS];
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
          a[m][j] = fp8_to_bf16(chunk_of(la, wm * 64 + m * 16 + lo, 4 * (h + j) + hi));
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        Bf16x16 w[CHUNKS];
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
          w[j] = fp8_to_bf16(chunk_of(lw, frag_row<GATED>(wn, f) + lo, 4 * (h + j) + hi));
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          f32x4 p = {0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < CHUNKS; ++j) {
            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j].lo, a[m][j].lo, p, 0, 0, 0);
            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j].hi, a[m][j].hi, p, 0, 0, 0);
          }
          const float sc = as[m] * ws[!GATED || f < 4 ? 0 : f - 4 < edge ? 1 : 2];
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][f][r] = __builtin_fmaf(sc, p[r], acc[m][f][r]);
        }
        if (!GATED) __builtin_amdgcn_sched_barrier(0);  // fragments in turn, for the registers
      }
    }
  }
}

// One tile: rows [row0, row0 + rows) of expert e, output columns [col0, col0 +
// cols). An expert's tiles go four tile columns at a time, all its row tiles.
struct Tile {
  int e, rows, col0, cols;
  int64_t row0;
};
template <int COLS>
__device__ __forceinline__ Tile tile_at(const GemmParams& P, const uint32_t* pre, uint64_t t, int across) {
  Tile o;
  o.e = expert_of_tile(pre, P.num_experts, (uint32_t)(t / across));
  const uint32_t first = (uint32_t)__builtin_amdgcn_readfirstlane((int)pre[o.e]);
  const uint32_t down = (uint32_t)__builtin_amdgcn_readfirstlane((int)pre[o.e + 1]) - first;
  const uint64_t in_e = t - (uint64_t)first * across;
  const int group = (int)(in_e / (4ull * down));
  const int wide = across - 4 * group < 4 ? across - 4 * group : 4;
  const int in_g = (int)(in_e - 4ull * down * group);
  const int rt = in_g / wide, ct = 4 * group + in_g % wide;
  const int left = rows_of(P, pre, o.e) - rt * kTile;
  o.rows = left < kTile ? left : kTile;
  o.row0 = (int64_t)o.e * P.max_tokens + (int64_t)rt * kTile;
  o.col0 = ct * COLS;
  o.cols = P.n - o.col0 < COLS ? P.n - o.col0 : COLS;
  return o;
}

template <int WEIGHT, bool GATED, bool OUT_FP8>
__global__ void __launch_bounds__(kThreads, 2) gemm_tile_kernel(const GemmParams P, int most) {
  extern __shared__ __align__(16) uint8_t lds_raw[];
  __shared__ uint32_t scan[kThreads / 64];
  __shared__ __align__(16) uint8_t step0[2 * kHalf];
  __shared__ __align__(16) uint8_t step1[2 * kHalf];
  uint32_t* pre = reinterpret_cast<uint32_t*>(lds_raw);
  tile_prefix<kThreads>(P, pre, scan, [=](int rows) { return big_tiles(rows, most); });
  const int tid = threadIdx.x, lane = tid & 63, lo = lane & 15, hi = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  constexpr int COLS = GATED ? 128 : 256;  // output columns of a tile
  const int across = (P.n + COLS - 1) / COLS;
  const uint32_t row_tiles = (uint32_t)__builtin_amdgcn_readfirstlane((int)pre[P.num_experts]);
  const uint64_t tiles = (uint64_t)row_tiles * across;
  constexpr bool FP8 = WEIGHT == kWeightFp8;
  const uint32_t ld = (uint32_t)P.k * (FP8 ? 1 : 2);
  const int steps = (int)((ld + kStepBytes - 1) / kStepBytes);
  const int kb = P.k / 128;

  // Workgroups are dealt to the XCDs in turn; each XCD takes a run of the
  // tiles, in which neighbours share rows or weights.
  const uint64_t x = blockIdx.x % kXcds, per = gridDim.x / kXcds;
  const uint64_t t0 = tiles * x / kXcds, t1 = tiles * (x + 1) / kXcds;
  for (uint64_t t = t0 + blockIdx.x / kXcds; t < t1; t += per) {
    const Tile tile = tile_at<COLS>(P, pre, t, across);
    const int e = tile.e, rows = tile.rows, col0 = tile.col0, cols = tile.cols;
    const int64_t row0 = tile.row0;

    Source s;
    s.ld = ld;
    s.a = rsrc_of(P.a + (uint64_t)row0 * ld, (uint32_t)rows * ld);
    const uint64_t w_row = (uint64_t)e * (GATED ? 2 : 1) * P.n + col0;
    // gated: wavefronts 4-7 copy the up rows
    const bool up = GATED && wave >= 4;
    s.w = rsrc_of(P.w + (w_row + (up ? P.n : 0)) * ld, (uint32_t)cols * ld);
    const uint32_t r = (uint32_t)wave * 32 + (lane >> 3);
    s.chunk = (uint32_t)((lane & 7) ^ (r & 7)) * 16;
    s.a_off = r * ld;
    s.w_off = (up ? r - 128 : r) * ld;

    // fp8 scales: this lane's four rows, and the tile's weight blocks
    const Rsrc ra = rsrc_of(FP8 ? P.a_scales + (uint64_t)row0 * kb : nullptr, FP8 ? (uint32_t)rows * kb * 4u : 0u);
    const int wrows = (GATED ? 2 : 1) * P.n;
    const float* wsp = FP8 ? static_cast<const float*>(P.w_scales) + (uint64_t)e * ((wrows + 127) / 128) * kb : nullptr;
    // the weight blocks of this wavefront's fragments: 128 rows at a multiple
    // of 128 (64 gate rows of them) lie in one; the 64 up rows start at any
    // multiple of 16, and from fragment `edge` on they lie in the next
    float as[2][4], ws[2][3];
    const int b0 = GATED ? (col0 + wn * 64) / 128 : (col0 + wn * 128) / 128;
    const int up0 = P.n + col0 + wn * 64;
    const int b1 = GATED ? up0 / 128 : b0;
    const int edge = ((b1 + 1) * 128 - up0) / 16;
    auto scales = [&](int step, float (&av)[4], float (&wv)[3]) {
      if constexpr (FP8) {
#pragma unroll
        for (int m = 0; m < 4; ++m)
          av[m] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
              ra, (int)(4u * ((uint32_t)(wm * 64 + m * 16 + lo) * kb + step)), 0, 0));
        const int last = (wrows + 127) / 128 - 1;
        wv[0] = wsp[(uint64_t)(b0 < last ? b0 : last) * kb + step];
        if constexpr (GATED) {
          wv[1] = wsp[(uint64_t)(b1 < last ? b1 : last) * kb + step];
          wv[2] = wsp[(uint64_t)(b1 < last ? b1 + 1 : last) * kb + step];
        }
      }
    };

    f32x4 acc[4][8];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int f = 0; f < 8; ++f) acc[m][f] = f32x4{0, 0, 0, 0};
    const bool busy = wm * 64 < rows;

    copy_step(s, 0, step0, wave);
    scales(0, as[0], ws[0]);
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    __syncthreads();
    for (int k = 0; k < steps; k += 2) {
      if (k + 1 < steps) {
        copy_step(s, k + 1, step1, wave);
        scales(k + 1, as[1], ws[1]);
      }
      if (busy) multiply<WEIGHT, GATED>(step0, wm, wn, as[0], ws[0], edge, acc);
      __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
      __syncthreads();
      if (k + 1 >= steps) break;
      if (k + 2 < steps) {
        copy_step(s, k + 2, step0, wave);
        scales(k + 2, as[0], ws[0]);
      }
      if (busy) multiply<WEIGHT, GATED>(step1, wm, wn, as[1], ws[1], edge, acc);
      __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
      __syncthreads();
    }

    // outputs: a lane's four consecutive columns of one row
    constexpr int F = GATED ? 4 : 8;
    float* amaxes = reinterpret_cast<float*>(step0);  // fp8: amax of a row's half, [256][2]
    if constexpr (GATED) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[m][f][q] = silu_mul(acc[m][f][q], acc[m][f + 4][q]);
    }
    if constexpr (OUT_FP8) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        float v = 0.0f;
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
          for (int q = 0; q < 4; ++q) v = fmaxf(v, fabsf(acc[m][f][q]));  // NaN is ignored
        v = fmaxf(v, __shfl_xor(v, 16, 64));
        v = fmaxf(v, __shfl_xor(v, 32, 64));
        if (hi == 0) amaxes[(wm * 64 + m * 16 + lo) * 2 + wn] = v;
      }
      __syncthreads();
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int row = wm * 64 + m * 16 + lo;
      if (row < rows) {
        const uint64_t orow = (uint64_t)(row0 + row);
        float inv = 0.0f;
        if constexpr (OUT_FP8) {
          const BlockScale s = block_scale(fmaxf(amaxes[row * 2], amaxes[row * 2 + 1]));
          inv = s.inv;
          if (wn == 0 && hi == 0) P.out_scales[orow * (P.n / 128) + col0 / 128] = s.scale;
        }
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const int col = wn * F * 16 + f * 16 + 4 * hi;
          const f32x4 v = acc[m][f];
          if (col < cols) {
            if constexpr (OUT_FP8)
              *reinterpret_cast<uint32_t*>(P.out + orow * P.n + col0 + col) =
                  e4m3_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
            else
              *reinterpret_cast<uint2*>(P.out + 2 * (orow * P.n + col0 + col)) =
                  make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
          }
        }
      }
    }
    __syncthreads();  // the buffers are free for the next tile
  }
}

// The same tiles with 4-bit weights. A k step is 64 columns: 32 KiB of A and
// 8 KiB of codes. The sums of a step (of half a step for groups of 32) are
// scaled and added up as gemm_few.h does; sum x comes from one product with
// ones a fragment of rows. Scales and zero points of the tile's 256 weight rows
// come in blocks of 8 groups into a ring of four blocks a row: a window of 8
// groups reads two of them, starting anywhere in the first, while the block
// behind the next window's first is written.
constexpr int kRing = 80, kZeroRing = 40;  // LDS bytes of a row, spread over the banks

template <int G, bool GATED>
__global__ void __launch_bounds__(kThreads, 2) gemm_tile_int4_kernel(const GemmParams P, int most) {
  extern __shared__ __align__(16) uint8_t lds_raw[];
  __shared__ uint32_t scan[kThreads / 64];
  __shared__ __align__(16) uint8_t a0[kHalf], a1[kHalf], w0[kTile * 32], w1[kTile * 32];
  __shared__ __align__(16) uint8_t ring[kTile * (kRing + kZeroRing)];
  uint32_t* pre = reinterpret_cast<uint32_t*>(lds_raw);
  tile_prefix<kThreads>(P, pre, scan, [=](int rows) { return big_tiles(rows, most); });
  const int tid = threadIdx.x, lane = tid & 63, lo = lane & 15, hi = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  constexpr int COLS = GATED ? 128 : 256;
  constexpr int GROUPS = G == 32 ? 2 : 1;  // sums of a step that are scaled apart
  const int across = (P.n + COLS - 1) / COLS;
  const uint32_t row_tiles = (uint32_t)__builtin_amdgcn_readfirstlane((int)pre[P.num_experts]);
  const uint64_t tiles = (uint64_t)row_tiles * across;
  const uint32_t lda = (uint32_t)P.k * 2, ldw = (uint32_t)P.k / 2;
  const int steps = (P.k + 63) / 64, groups = P.k / G;
  const int rows_w = (GATED ? 2 : 1) * P.n;
  const uint32_t values = (uint32_t)rows_w * groups;
  const float z_none = P.w_zeros ? 16.0f : 24.0f;
  const CodeMasks masks;
  const v4u one = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const bf16x8 ones = __builtin_bit_cast(bf16x8, one);
  const f32x4 zero = {0, 0, 0, 0};

  const uint64_t x = blockIdx.x % kXcds, per = gridDim.x / kXcds;
  const uint64_t t0 = tiles * x / kXcds, t1 = tiles * (x + 1) / kXcds;
  for (uint64_t t = t0 + blockIdx.x / kXcds; t < t1; t += per) {
    const Tile tile = tile_at<COLS>(P, pre, t, across);
    const int rows = tile.rows, col0 = tile.col0, cols = tile.cols;
    const Rsrc ra = rsrc_of(P.a + (uint64_t)tile.row0 * lda, (uint32_t)rows * lda);
    const uint64_t w_row = (uint64_t)tile.e * rows_w + col0;
    const bool up = GATED && wave >= 4;  // wavefronts 4-7 copy the up rows
    const Rsrc rw = rsrc_of(P.w + (w_row + (up ? P.n : 0)) * ldw, (uint32_t)cols * ldw);
    const uint32_t ar = (uint32_t)wave * 32 + (lane >> 3), achunk = (uint32_t)((lane & 7) ^ (ar & 7)) * 16;
    // codes: 32 rows an instruction, two lanes a row; a row's halves change
    // places with bit 3 of the row, for the banks
    const uint32_t wr = (uint32_t)wave * 32 + (lane >> 1);
    const uint32_t whalf = (uint32_t)((lane & 1) ^ (wr >> 3 & 1)) * 16;
    const uint32_t w_off = (up ? wr - 128 : wr) * ldw;
    auto copy = [&](int step, uint8_t* ta, uint8_t* tw) {
      const uint32_t at = (uint32_t)step * 128 + achunk;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            ra, (LdsByte*)(ta + (wave * 32 + i * 8) * kStepBytes), 16,
            at < lda ? (int)((ar + i * 8) * lda + at) : (int)kOutside, 0, 0, 0);
      const uint32_t wat = (uint32_t)step * 32 + whalf;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (LdsByte*)(tw + wave * 32 * 32), 16,
                                               wat < ldw ? (int)(w_off + wat) : (int)kOutside, 0, 0, 0);
    };

    // the ring: thread i < 256 brings in tile row i's blocks
    const Rsrc rs = rsrc_of(static_cast<const uint16_t*>(P.w_scales) + (uint64_t)tile.e * values, 2 * values);
    const Rsrc rz = rsrc_of(P.w_zeros + (P.w_zeros ? (uint64_t)tile.e * values : 0), P.w_zeros ? values : 0u);
    auto weight_row = [&](int i) { return col0 + (GATED && i >= 128 ? P.n + i - 128 : i); };
    uint32_t block = 2 * (uint32_t)weight_row(tid & 255) * groups & ~15u;
    uint32_t zblock = (uint32_t)weight_row(tid & 255) * groups & ~7u;
    v4u next = {0, 0, 0, 0};
    v2u znext = {0, 0};
    auto fetch = [&] {
      next = __builtin_amdgcn_raw_buffer_load_b128(rs, (int)block, 0, 0);
      znext = __builtin_amdgcn_raw_buffer_load_b64(rz, (int)zblock, 0, 0);
      block += 16;
      zblock += 8;
    };
    auto put = [&](int b) {
      *reinterpret_cast<v4u*>(ring + tid * kRing + (b & 3) * 16) = next;
      *reinterpret_cast<v2u*>(ring + kTile * kRing + tid * kZeroRing + (b & 3) * 8) = znext;
    };
    // rows 16 apart start alike in their blocks, and n, a multiple of 8, apart
    const uint32_t phase = (uint32_t)(lo * groups) & 7;
    const uint8_t* ring_at = ring + lo * kRing;
    const uint8_t* zring_at = ring + kTile * kRing + lo * kZeroRing;

    f32x4 acc[4][8];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int f = 0; f < 8; ++f) acc[m][f] = zero;
    const bool busy = wm * 64 < rows;

    auto multiply4 = [&](int step, const uint8_t* la, const uint8_t* lw) __attribute__((always_inline)) {
      bf16x8 a[4][2];
      f32x4 sum[4][GROUPS];
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          a[m][j] = a_like_codes(chunk_of(la, wm * 64 + m * 16 + lo, 4 * j + hi));
          const int u = GROUPS == 2 ? j : 0;
          sum[m][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              a[m][j], ones, GROUPS == 2 || j == 0 ? zero : sum[m][u], 0, 0, 0);
        }
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        const int r = frag_row<GATED>(wn, f) + lo;
#pragma unroll
        for (int u = 0; u < GROUPS; ++u) {
          f32x4 p[4];
#pragma unroll
          for (int j = u; j < (GROUPS == 2 ? u + 1 : 2); ++j) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(lw + r * 32 + ((j ^ (r >> 3 & 1)) << 4) + hi * 4);
            const bf16x8 wf = codes_bf16(w, masks);
#pragma unroll
            for (int m = 0; m < 4; ++m)
              p[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[m][j], wf, j == u ? zero : p[m], 0, 0, 0);
          }
          const int g = G == 128 ? step >> 1 : step * GROUPS + u;
          const uint32_t at = phase + (uint32_t)g;
          const int row = frag_row<GATED>(wn, f);
          const float read = __uint_as_float(
              (uint32_t) * reinterpret_cast<const uint16_t*>(ring_at + 2 * (at & 31) + row * kRing) << 16);
          const float sc = G == 128 || g < groups ? read : 0.0f;
          const float off = z_none + (float)zring_at[(at & 31) + row * kZeroRing];
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              acc[m][f][q] = __builtin_fmaf(sc, __builtin_fmaf(-off, sum[m][u][q], p[m][q]), acc[m][f][q]);
        }
        if (f & 1) __builtin_amdgcn_sched_barrier(0);  // fragments in turn, for the registers
      }
    };
    // a window of 8 groups starts: the block behind the next window's first
    constexpr int WINDOW = 8 * G / 64;  // steps
    auto enter = [&](int step) {
      if (step % WINDOW == 0 && wave < 4) {
        put(step / WINDOW + 2);
        fetch();
      }
    };

    copy(0, a0, w0);
    if (wave < 4) {
      fetch();
      put(0);
      fetch();
      put(1);
      fetch();
    }
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    __syncthreads();
    for (int k = 0; k < steps; k += 2) {
      enter(k);
      if (k + 1 < steps) copy(k + 1, a1, w1);
      if (busy) multiply4(k, a0, w0);
      __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
      __syncthreads();
      if (k + 1 >= steps) break;
      if (k + 2 < steps) copy(k + 2, a0, w0);
      if (busy) multiply4(k + 1, a1, w1);
      __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
      __syncthreads();
    }

    // outputs: 16 rows of a wavefront pass through LDS, four columns a lane
    constexpr int F = GATED ? 4 : 8, LD = F * 16;
    static_assert(4 * 16 * LD * 4 <= kHalf, "four wavefronts a buffer");
    float* mine = reinterpret_cast<float*>(wave < 4 ? a0 : a1) + (wave & 3) * 16 * LD;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v = acc[m][f][q];
          if constexpr (GATED) v = silu_mul(v, acc[m][f + 4][q]);
          mine[(4 * hi + q) * LD + f * 16 + lo] = v;
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = lane; i < 16 * F * 4; i += 64) {
        const int r = i / (F * 4), c = 4 * (i % (F * 4)), row = wm * 64 + m * 16 + r;
        const int col = wn * F * 16 + c;
        const f32x4 v = *reinterpret_cast<const f32x4*>(mine + r * LD + c);
        if (row < rows && col < cols)
          *reinterpret_cast<uint2*>(P.out + 2 * ((uint64_t)(tile.row0 + row) * P.n + col0 + col)) =
              make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();  // the buffers are free for the next tile
  }
}

template <int G>
hipError_t launch_int4(const GemmParams& p, int most, hipStream_t stream) {
  const uint32_t lds = tile_prefix_bytes(p.num_experts);
  if (p.gated) gemm_tile_int4_kernel<G, true><<<256, kThreads, lds, stream>>>(p, most);
  else gemm_tile_int4_kernel<G, false><<<256, kThreads, lds, stream>>>(p, most);
  return hipGetLastError();
}

template <int WEIGHT, bool GATED, bool OUT_FP8>
hipError_t launch(const GemmParams& p, int most, hipStream_t stream) {
  gemm_tile_kernel<WEIGHT, GATED, OUT_FP8>
      <<<256, kThreads, tile_prefix_bytes(p.num_experts), stream>>>(p, most);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_tile(const GemmParams& p, int most, hipStream_t stream) {
  if (p.weight == kWeightFp8) {
    if (p.out_fp8) return launch<kWeightFp8, true, true>(p, most, stream);
    return p.gated ? launch<kWeightFp8, true, false>(p, most, stream)
                   : launch<kWeightFp8, false, false>(p, most, stream);
  }
  if (p.weight == kWeightInt4)
    return p.group == 128  ? launch_int4<128>(p, most, stream)
           : p.group == 64 ? launch_int4<64>(p, most, stream)
                           : launch_int4<32>(p, most, stream);
  return p.gated ? launch<kWeightBf16, true, false>(p, most, stream)
                 : launch<kWeightBf16, false, false>(p, most, stream);
}

}  // namespace llmoe
