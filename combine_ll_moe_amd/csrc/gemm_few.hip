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
constexpr int kFewFrags = 4;      // weight strips a wavefront holds at once
constexpr int kFewWaves = 4;      // of a workgroup
// From this many strips a wavefront (in units of what it holds at once) on,
// the list is long.
constexpr int kFewLong = 4;
// LDS of a workgroup: partial sums, or the wavefronts' rings of scales and
// the two steps' rows of A.
constexpr int kRingBytes = 64 * 72;
constexpr int kPoolBytes = kFewWaves * kRingBytes + 2 * kFewRows * 256;

__device__ __forceinline__ Rsrc rsrc_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, kBufferWord3);
}
__device__ __forceinline__ v4u load16(Rsrc r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
}

__device__ __forceinline__ float load_f32(Rsrc r, uint32_t off) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
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
  constexpr int D = MF + NF <= 5 ? 4 : MF + NF <= 6 ? 3 : 2;  // chunks in flight
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
      __builtin_amdgcn_sched_barrier(0);  // a stage waits for its own loads, not for the next one's
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
  // Those of a chunk behind k are zeros.
  const Rsrc rs = rsrc_of(it.a_scales, (uint32_t)it.rows * chunks * 4u);
  const Rsrc rws = rsrc_of(static_cast<const float*>(P.w_scales) + (uint64_t)it.e * blocks * chunks,
                           (uint32_t)blocks * chunks * 4u);
  const uint32_t as_at = 4u * ((MF > 1 ? hi % MF : 0) * 16 + lo) * chunks;
  const uint32_t ws_at = 4u * (strip_row<NF, GATED>(P, it.strip, hi % NF) / 128) * chunks;
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
    as[s] = load_f32(rs, in ? as_at + 4u * c : kOutside);
    sw[s] = load_f32(rws, in ? ws_at + 4u * c : kOutside);
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
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        const float av = MF > 1 ? __shfl(as[s], m * 16 + lo, 64) : as[s];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          const float wv = __builtin_bit_cast(
              float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sw[s]), f * 16));
          const float sc = av * wv;
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][f][r] = __builtin_fmaf(sc, p[m][f][r], acc[m][f][r]);
        }
      }
      load(s, c + (s + D) * WK);
      __builtin_amdgcn_sched_barrier(0);  // a stage waits for its own loads, not for the next one's
    }
  }
}

// Four words of four lane quarters transposed: word j of quarter q becomes
// word q of quarter j.
__device__ __forceinline__ void transpose_quarters(uint32_t (&w)[4]) {
  auto swap32 = [](uint32_t& a, uint32_t& b) {
    const auto v = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = v[0];
    b = v[1];
  };
  auto swap16 = [](uint32_t& a, uint32_t& b) {
    const auto v = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = v[0];
    b = v[1];
  };
  swap32(w[0], w[2]);
  swap32(w[1], w[3]);
  swap16(w[0], w[1]);
  swap16(w[2], w[3]);
}

// A wavefront's int4 scales and zero points. A group's value of 64 weight rows
// lies in 64 cache lines, so loads a group at a time would ask the caches for
// as much as the codes do; here a lane takes the next 16 bytes (8 groups) of
// one row's scales and 8 of its zero points, whole aligned blocks, into a
// ring of two blocks a row in LDS, and every lane reads its rows' values from
// there. A row starts anywhere in a block: a window of 8 groups touches two.
template <int NF, bool GATED>
struct ScaleRing {
  static constexpr int kRow = 48, kZeroRow = 24;  // LDS bytes of a row, spread over the banks
  static constexpr int kBytes = 64 * (kRow + kZeroRow);
  Rsrc rs, rz;
  uint8_t* lds;
  uint32_t block, zblock;       // this lane's next block's offset
  v4u next;
  v2u znext;
  uint32_t at[NF], zat[NF];     // LDS: row f * 16 + lane % 16
  uint32_t phase[NF], zphase[NF];
  float none;
  static_assert(kBytes <= kRingBytes);

  __device__ __forceinline__ void init(const GemmParams& P, const Item& it, int groups, int first,
                                       uint8_t* ring) {
    const int lane = threadIdx.x & 63, lo = lane & 15, hi = lane >> 4;
    const int rows_w = (GATED ? 2 : 1) * P.n;
    const uint32_t values = (uint32_t)rows_w * groups;
    rs = rsrc_of(static_cast<const uint16_t*>(P.w_scales) + (uint64_t)it.e * values, 2 * values);
    // without zero points their descriptor is empty
    rz = rsrc_of(P.w_zeros + (P.w_zeros ? (uint64_t)it.e * values : 0), P.w_zeros ? values : 0u);
    none = P.w_zeros ? 16.0f : 24.0f;
    lds = ring;
    const uint32_t g0 = (uint32_t)(strip_row<NF, GATED>(P, it.strip, hi % NF) + lo) * groups + first;
    block = 2 * g0 & ~15u;
    zblock = g0 & ~7u;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const uint32_t g = (uint32_t)(strip_row<NF, GATED>(P, it.strip, f) + lo) * groups + first;
      at[f] = (f * 16 + lo) * kRow;
      zat[f] = 64 * kRow + (f * 16 + lo) * kZeroRow;
      phase[f] = 2 * g & 15;
      zphase[f] = g & 7;
    }
    fetch();
    put(0);
    fetch();
    put(1);
    fetch();
  }
  __device__ __forceinline__ void fetch() {
    next = load16(rs, block);
    znext = __builtin_amdgcn_raw_buffer_load_b64(rz, (int)zblock, 0, 0);
    block += 16;
    zblock += 8;
  }
  __device__ __forceinline__ void put(int slot) {
    const int lane = threadIdx.x & 63;
    *reinterpret_cast<v4u*>(lds + lane * kRow + slot * 16) = next;
    *reinterpret_cast<v2u*>(lds + 64 * kRow + lane * kZeroRow + slot * 8) = znext;
  }
  // Before group g (from `first`) is read: at a window's start the block
  // behind it comes in, in the place of the one before it.
  __device__ __forceinline__ void enter(int g) {
    if (g > 0 && g % 8 == 0) {
      put((g / 8 + 1) & 1);
      fetch();
    }
  }
  __device__ __forceinline__ float scale(int f, int g) const {
    return __uint_as_float(
        (uint32_t) * reinterpret_cast<const uint16_t*>(lds + at[f] + ((phase[f] + 2 * g) & 31)) << 16);
  }
  __device__ __forceinline__ float zero(int f, int g) const {
    return none + (float)lds[zat[f] + ((zphase[f] + g) & 15)];
  }
};

// A chunk is 128 columns: 16 bytes of codes a lane, quarter q the columns
// [32 q, 32 q + 32). Transposed among the quarters, word j of quarter q holds
// columns 32 j + 8 q and on: product j covers columns [32 j, 32 j + 32), which
// lie in one group, and A's fragments are read as they stand.
template <int MF, int NF, bool GATED, int G>
__device__ __forceinline__ void sum_int4(const GemmParams& P, const Item& it, int kw, int WK,
                                         uint8_t* ring_lds, f32x4 (&acc)[MF][NF]) {
  constexpr int D = MF == 4 ? 1 : MF == 2 ? 2 : 3;
  constexpr int GROUPS = 128 / G;  // of a chunk
  const int lane = threadIdx.x & 63;
  const uint32_t lda = 2u * (uint32_t)P.k, ldw = (uint32_t)P.k / 2;
  const int groups = P.k / G, chunks = (P.k + 127) / 128;
  // a run of chunks for each wavefront, for its ring of scales
  const int c0 = chunks * kw / WK, c1 = chunks * (kw + 1) / WK;
  const Rsrc ra = rsrc_of(it.a, (uint32_t)it.rows * lda);
  Rsrc rw[NF];
  const int rows_w = (GATED ? 2 : 1) * P.n;
#pragma unroll
  for (int f = 0; f < NF; ++f)
    rw[f] = rsrc_of(P.w + ((uint64_t)it.e * rows_w + strip_row<NF, GATED>(P, it.strip, f)) * ldw,
                    (uint32_t)strip_rows<NF, GATED>(P, it, f) * ldw);
  const uint32_t lo = lane & 15, hi = lane >> 4;
  ScaleRing<NF, GATED> ring;
  v4u wb[D][NF], ab[D][MF][4];
  auto load = [&](int s, int c) {
    const uint32_t wat = 64u * (uint32_t)c + 16u * hi;
    const uint32_t woff = c < c1 && wat < ldw ? lo * ldw + wat : kOutside;
#pragma unroll
    for (int f = 0; f < NF; ++f) wb[s][f] = load16(rw[f], woff);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t at = 256u * (uint32_t)c + 64u * j + 16u * hi;
      const bool in = c < c1 && at < lda;
#pragma unroll
      for (int m = 0; m < MF; ++m)
        ab[s][m][j] = load16(ra, in ? (lo + m * 16u) * lda + at : kOutside);
    }
  };
  const v4u one = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const bf16x8 ones = __builtin_bit_cast(bf16x8, one);
  const CodeMasks masks;
#pragma unroll
  for (int s = 0; s < D; ++s) load(s, c0 + s);
  ring.init(P, it, groups, c0 * GROUPS, ring_lds);
  for (int c = c0; c < c1; c += D) {
#pragma unroll
    for (int s = 0; s < D; ++s) {
      if (c + s >= c1) break;
      const f32x4 zero = {0, 0, 0, 0};
      uint32_t wt[NF][4];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        wt[f][0] = wb[s][f].x, wt[f][1] = wb[s][f].y, wt[f][2] = wb[s][f].z, wt[f][3] = wb[s][f].w;
        transpose_quarters(wt[f]);
      }
      ring.enter((c + s - c0) * GROUPS);
#pragma unroll
      for (int u = 0; u < GROUPS; ++u) {
        const int g = (c + s) * GROUPS + u;
        f32x4 p[MF][NF], sum[MF];
#pragma unroll
        for (int j = u * (G / 32); j < (u + 1) * (G / 32); ++j) {
          const bool start = j == u * (G / 32);
          bf16x8 x[MF];
#pragma unroll
          for (int m = 0; m < MF; ++m) {
            x[m] = a_like_codes(ab[s][m][j]);
            sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[m], ones, start ? zero : sum[m], 0, 0, 0);
          }
#pragma unroll
          for (int f = 0; f < NF; ++f) {
            const bf16x8 wf = codes_bf16(wt[f][j], masks);
#pragma unroll
            for (int m = 0; m < MF; ++m)
              p[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[m], wf, start ? zero : p[m][f], 0, 0, 0);
          }
        }
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          // a group behind k is zeros, times what may be a NaN: scale 0
          const float read = ring.scale(f, g - c0 * GROUPS);
          const float sc = g < groups ? read : 0.0f;
          const float off = ring.zero(f, g - c0 * GROUPS);
#pragma unroll
          for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[m][f][r] = __builtin_fmaf(sc, __builtin_fmaf(-off, sum[m][r], p[m][f][r]), acc[m][f][r]);
        }
        __builtin_amdgcn_sched_barrier(0);  // groups in turn: their registers do not add up
      }
      load(s, c + s + D);
    }
  }
}

// The long list's form: the four wavefronts of a workgroup take strips beside
// each other over all of k and share the rows of A through LDS. W still goes
// straight into registers, D steps ahead; a step's A goes through registers,
// also D steps ahead (a wait for a load waits for every older one too, so
// both have to be ordered alike), and is written to LDS as the products read
// it: as bf16, for int4 in the order of the codes.
template <int WEIGHT>
constexpr int step_columns = WEIGHT == kWeightBf16 ? 64 : 128;

template <int WEIGHT, int G, int MF, int NF, bool GATED>
__device__ __forceinline__ void sum_shared(const GemmParams& P, const Item& it, const Item& mine,
                                           uint8_t* abuf, uint8_t* ring_lds,
                                           f32x4 (&acc)[MF][NF]) {
  constexpr bool FP8 = WEIGHT == kWeightFp8, INT4 = WEIGHT == kWeightInt4;
  constexpr int KS = step_columns<WEIGHT>;
  constexpr int ROW = 2 * KS;                       // LDS bytes of a row of a step
  constexpr int STEP = MF * 16 * ROW;
  constexpr int CH = ROW / 16;                      // 16-byte chunks of it
  constexpr int D = MF == 4 ? 2 : 3;
  constexpr int A_ITEM = FP8 ? 1 : 2;               // bytes of a value of A in memory
  constexpr int A_CH = KS * A_ITEM / 16;            // 16-byte loads of a row
  constexpr int AL = (MF * 16 * A_CH + 255) / 256;  // loads of a thread
  constexpr int WL = KS * (FP8 ? 2 : INT4 ? 1 : 4) / 128;  // 16-byte loads of a strip
  constexpr int GROUPS = INT4 ? 128 / G : 1;
  const int tid = threadIdx.x, lane = tid & 63, lo = lane & 15, hi = lane >> 4;
  const int steps = (P.k + KS - 1) / KS;
  const uint32_t lda = (uint32_t)P.k * A_ITEM;
  const uint32_t ldw = INT4 ? (uint32_t)P.k / 2 : lda;
  const Rsrc ra = rsrc_of(it.a, (uint32_t)it.rows * lda);
  const int rows_w = (GATED ? 2 : 1) * P.n;
  Rsrc rw[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
    rw[f] = rsrc_of(P.w + ((uint64_t)it.e * rows_w + strip_row<NF, GATED>(P, mine.strip, f)) * ldw,
                    (uint32_t)strip_rows<NF, GATED>(P, mine, f) * ldw);

  // Scales. fp8: lane quarter q loads row fragment q's and strip q's; those
  // behind k are zeros. int4: a ring.
  const int groups = INT4 ? P.k / G : steps, blocks = (rows_w + 127) / 128;
  const Rsrc rs = rsrc_of(static_cast<const float*>(P.w_scales) + (FP8 ? (uint64_t)it.e * blocks * groups : 0),
                          FP8 ? 4u * blocks * groups : 0u);
  const Rsrc ras = rsrc_of(it.a_scales, FP8 ? (uint32_t)it.rows * groups * 4u : 0u);
  const uint32_t s_at = 4u * (strip_row<NF, GATED>(P, mine.strip, hi % NF) / 128) * groups;
  const uint32_t as_at = 4u * ((MF > 1 ? hi % MF : 0) * 16 + lo) * groups;
  ScaleRing<NF, GATED> ring;

  v4u wb[D][NF][WL], ab[D][AL];
  float as[D], sw[D];
  auto load_a = [&](int s, int step) {
#pragma unroll
    for (int i = 0; i < AL; ++i) {
      const int q = tid + 256 * i, row = q / A_CH;
      const uint32_t at = (uint32_t)step * (KS * A_ITEM) + 16u * (q % A_CH);
      const bool in = step < steps && at < lda && row < MF * 16;
      ab[s][i] = load16(ra, in ? (uint32_t)row * lda + at : kOutside);
    }
  };
  auto store_a = [&](int s, int step) {
    uint8_t* to = abuf + (step & 1) * STEP;
#pragma unroll
    for (int i = 0; i < AL; ++i) {
      const int q = tid + 256 * i, row = q / A_CH, c = q % A_CH;
      if (MF * 16 * A_CH % 256 && row >= MF * 16) break;
      uint8_t* r = to + row * ROW;
      if constexpr (FP8) {
        const Bf16x16 v = fp8_to_bf16(ab[s][i]);
        *reinterpret_cast<bf16x8*>(r + (((2 * c) ^ row) & (CH - 1)) * 16) = v.lo;
        *reinterpret_cast<bf16x8*>(r + (((2 * c + 1) ^ row) & (CH - 1)) * 16) = v.hi;
      } else if constexpr (INT4) {
        *reinterpret_cast<bf16x8*>(r + ((c ^ row) & (CH - 1)) * 16) = a_like_codes(ab[s][i]);
      } else {
        *reinterpret_cast<v4u*>(r + ((c ^ row) & (CH - 1)) * 16) = ab[s][i];
      }
    }
  };
  auto load_w = [&](int s, int step) {
#pragma unroll
    for (int j = 0; j < WL; ++j) {
      const uint32_t at = (uint32_t)step * (64 * WL) + 64u * j + 16u * hi;
      const uint32_t off = step < steps && at < ldw ? lo * ldw + at : kOutside;
#pragma unroll
      for (int f = 0; f < NF; ++f) wb[s][f][j] = load16(rw[f], off);
    }
    if constexpr (FP8) {
      as[s] = load_f32(ras, step < steps ? as_at + 4u * step : kOutside);
      sw[s] = load_f32(rs, step < steps ? s_at + 4u * step : kOutside);
    }
  };
  const v4u one = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const bf16x8 ones = __builtin_bit_cast(bf16x8, one);
  const CodeMasks masks;
  const f32x4 zero = {0, 0, 0, 0};
  auto multiply = [&](int s, int step) __attribute__((always_inline)) {
    const uint8_t* from = abuf + (step & 1) * STEP;
    auto a_chunk = [&](int m, int c) {
      const int row = m * 16 + lo;
      return *reinterpret_cast<const bf16x8*>(from + row * ROW + ((c ^ row) & (CH - 1)) * 16);
    };
    if constexpr (WEIGHT == kWeightBf16) {
#pragma unroll
      for (int j = 0; j < WL; ++j)
#pragma unroll
        for (int m = 0; m < MF; ++m) {
          const bf16x8 a = a_chunk(m, 4 * j + hi);
#pragma unroll
          for (int f = 0; f < NF; ++f)
            acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                a, __builtin_bit_cast(bf16x8, wb[s][f][j]), acc[m][f], 0, 0, 0);
        }
    } else if constexpr (FP8) {
      float av[MF];
#pragma unroll
      for (int m = 0; m < MF; ++m) av[m] = MF > 1 ? __shfl(as[s], m * 16 + lo, 64) : as[s];
      constexpr int FB = MF == 4 ? 1 : NF;  // strips at a time
#pragma unroll
      for (int f0 = 0; f0 < NF; f0 += FB) {
        f32x4 p[MF][FB];
#pragma unroll
        for (int j = 0; j < WL; ++j) {
          Bf16x16 w[FB];
#pragma unroll
          for (int f = 0; f < FB; ++f) w[f] = fp8_to_bf16(wb[s][f0 + f][j]);
#pragma unroll
          for (int m = 0; m < MF; ++m) {
            const bf16x8 a0 = a_chunk(m, 8 * j + 2 * hi), a1 = a_chunk(m, 8 * j + 2 * hi + 1);
#pragma unroll
            for (int f = 0; f < FB; ++f) {
              p[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[f].lo, a0, j ? p[m][f] : zero, 0, 0, 0);
              p[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[f].hi, a1, p[m][f], 0, 0, 0);
            }
          }
        }
#pragma unroll
        for (int f = 0; f < FB; ++f) {
          const float wv = __builtin_bit_cast(
              float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sw[s]), (f0 + f) * 16));
#pragma unroll
          for (int m = 0; m < MF; ++m) {
            const float sc = av[m] * wv;
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[m][f0 + f][r] = __builtin_fmaf(sc, p[m][f][r], acc[m][f0 + f][r]);
          }
        }
        if (FB < NF) __builtin_amdgcn_sched_barrier(0);  // strips in turn, for the registers
      }
    } else {
      // Groups of 128: the word j of quarter q holds columns 32 q + 8 j and on,
      // and A is read to match. Smaller groups: transposed, see sum_int4.
      ring.enter(step * GROUPS);
      uint32_t wt[NF][4];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        wt[f][0] = wb[s][f][0].x, wt[f][1] = wb[s][f][0].y, wt[f][2] = wb[s][f][0].z, wt[f][3] = wb[s][f][0].w;
        if constexpr (G < 128) transpose_quarters(wt[f]);
      }
#pragma unroll
      for (int u = 0; u < GROUPS; ++u) {
        const int g = step * GROUPS + u;
        constexpr int FB = MF == 4 ? 1 : NF;
        f32x4 sum[MF];
#pragma unroll
        for (int f0 = 0; f0 < NF; f0 += FB) {
          f32x4 p[MF][FB];
#pragma unroll
          for (int j = u * (G / 32); j < (u + 1) * (G / 32); ++j) {
            const bool start = j == u * (G / 32);
            bf16x8 w[FB];
#pragma unroll
            for (int f = 0; f < FB; ++f) w[f] = codes_bf16(wt[f0 + f][j], masks);
#pragma unroll
            for (int m = 0; m < MF; ++m) {
              const bf16x8 a = a_chunk(m, G < 128 ? 4 * j + hi : 4 * hi + j);
              if (f0 == 0)
                sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, ones, start ? zero : sum[m], 0, 0, 0);
#pragma unroll
              for (int f = 0; f < FB; ++f)
                p[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, w[f], start ? zero : p[m][f], 0, 0, 0);
            }
          }
#pragma unroll
          for (int f = 0; f < FB; ++f) {
            // a group behind k is zeros, times what may be a NaN: scale 0
            const float read = ring.scale(f0 + f, g);
            const float sc = G == 128 || g < groups ? read : 0.0f;
            const float off = ring.zero(f0 + f, g);
#pragma unroll
            for (int m = 0; m < MF; ++m)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                acc[m][f0 + f][r] = __builtin_fmaf(
                    sc, __builtin_fmaf(-off, sum[m][r], p[m][f][r]), acc[m][f0 + f][r]);
          }
          if (FB < NF) __builtin_amdgcn_sched_barrier(0);  // strips in turn, for the registers
        }
        __builtin_amdgcn_sched_barrier(0);  // groups in turn: their registers do not add up
      }
    }
  };

  // ab[i] holds step i's rows of A (mod D), wb[i] its weights
#pragma unroll
  for (int s = 0; s < D; ++s) {
    load_a(s, s);
    load_w(s, s);
  }
  if constexpr (INT4) ring.init(P, mine, groups, 0, ring_lds);
  __syncthreads();  // the buffers' last reader is done
  store_a(0, 0);
  load_a(0, D);
  for (int k = 0; k < steps; k += D) {
#pragma unroll
    for (int s = 0; s < D; ++s) {
      const int step = k + s;
      if (step >= steps) break;  // the same for the whole workgroup
      __syncthreads();           // step's A is there, and the step before is read
      store_a((s + 1) % D, step + 1);
      load_a((s + 1) % D, step + 1 + D);
      multiply(s, step);
      load_w(s, step + D);
    }
  }
}

// One item. SPLIT: the wavefronts split k between them; else they take its
// strips beside each other. Sums first, then, 16 rows at a time, they pass
// through LDS and the outputs go out, four columns a thread.
template <int WEIGHT, int G, int MF, int NF, bool GATED, bool OUT_FP8, bool SPLIT>
__device__ __forceinline__ void do_item(const GemmParams& P, const Item& it, uint8_t* pool) {
  constexpr bool ALONE = !SPLIT && !OUT_FP8;  // a wavefront's outputs are its own
  constexpr int WN = OUT_FP8 ? kFewWaves : 1;
  constexpr int PARTS = SPLIT ? kFewWaves : 1;
  constexpr int SF = GATED ? NF / 2 : NF;   // output strips a wavefront
  constexpr int LD = NF * 16 + 4;           // floats of a partial row
  constexpr int COLS = WN * SF * 16;
  constexpr int THREADS = ALONE ? 64 : kFewWaves * 64;
  // row fragments that pass through LDS at once
  constexpr int FIT = kPoolBytes / (kFewWaves * 16 * LD * 4);
  constexpr int MP = FIT >= MF ? MF : FIT >= 2 ? 2 : 1;
  static_assert(FIT >= 1);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tid = ALONE ? lane : threadIdx.x;
  Item mine = it;
  if constexpr (!SPLIT) {
    const int s0 = it.strips * wave / kFewWaves;
    mine.strip = it.strip + s0;
    mine.strips = it.strips * (wave + 1) / kFewWaves - s0;
  }
  f32x4 acc[MF][NF];
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[m][f] = f32x4{0, 0, 0, 0};
  uint8_t* ring = pool + wave * kRingBytes;
  if constexpr (!SPLIT)
    sum_shared<WEIGHT, G, MF, NF, GATED>(P, it, mine, pool + kFewWaves * kRingBytes, ring, acc);
  else if constexpr (WEIGHT == kWeightBf16)
    sum_bf16<MF, NF, GATED>(P, mine, wave, kFewWaves, acc);
  else if constexpr (WEIGHT == kWeightFp8)
    sum_fp8<MF, NF, GATED>(P, mine, wave, kFewWaves, acc);
  else
    sum_int4<MF, NF, GATED, G>(P, mine, wave, kFewWaves, ring, acc);

  auto meet = [] {
    if constexpr (ALONE) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    } else {
      __syncthreads();
    }
  };
  // the pool was the rings' and A's until here
  if (!SPLIT || WEIGHT == kWeightInt4) __syncthreads();
  const int lo = lane & 15, hi = lane >> 4;
  constexpr int WAVE = MP * 16 * LD;
  float* part = reinterpret_cast<float*>(pool);
  float* mp = part + wave * WAVE;
  const float* first = ALONE ? mp : part;
#pragma unroll
  for (int m0 = 0; m0 < MF; m0 += MP) {
    if (m0 * 16 >= it.rows) break;  // the same for all who meet
#pragma unroll
    for (int m = 0; m < MP; ++m)
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        float* to = mp + m * 16 * LD + f * 16;
        if constexpr (WEIGHT == kWeightFp8) {
          *reinterpret_cast<f32x4*>(to + lo * LD + 4 * hi) = acc[m0 + m][f];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) to[(4 * hi + r) * LD + lo] = acc[m0 + m][f][r];
        }
      }
    meet();
    const int rows = it.rows - m0 * 16 < MP * 16 ? it.rows - m0 * 16 : MP * 16;
    // (fp8 out: whole wavefronts hold rows together, so none leaves early)
    const int todo = (OUT_FP8 ? MP * 16 : rows) * (COLS / 4);
    for (int i = tid; i < todo; i += THREADS) {
      const int row = i / (COLS / 4), c4 = 4 * (i % (COLS / 4));
      const int list = c4 / (SF * 16), at = c4 % (SF * 16);
      f32x4 v = {0, 0, 0, 0}, u = {0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < PARTS; ++q) {
        const float* p = first + (SPLIT ? q : list) * WAVE + row * LD + at;
        v += *reinterpret_cast<const f32x4*>(p);
        if constexpr (GATED) u += *reinterpret_cast<const f32x4*>(p + SF * 16);
      }
      if constexpr (GATED) {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = silu_mul(v[r], u[r]);
      }
      const Item& of = ALONE ? mine : it;
      const int col = of.strip * 16 + c4;
      const bool in = row < rows && col < P.n && c4 < of.strips * 16;
      const uint64_t orow = (uint64_t)(it.row0 + m0 * 16 + row);
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
  // before the next item's rings: a wavefront's part of the pool was not
  // where its ring is
  if (ALONE) __syncthreads();
}

template <int WEIGHT, int G, int NF, bool GATED, bool OUT_FP8, bool SPLIT>
__device__ __forceinline__ void do_item_rows(const GemmParams& P, const Item& it, uint8_t* pool) {
  if (it.rows <= 16) {
    do_item<WEIGHT, G, 1, NF, GATED, OUT_FP8, SPLIT>(P, it, pool);
  } else if (it.rows <= 32) {
    do_item<WEIGHT, G, 2, NF, GATED, OUT_FP8, SPLIT>(P, it, pool);
  } else if constexpr (SPLIT && WEIGHT != kWeightBf16 && NF == 4) {
    // registers hold 64 rows of A beside two strips
    constexpr int SF = GATED ? 1 : 2;
    Item half = it;
    half.strips = it.strips < SF ? it.strips : SF;
    do_item<WEIGHT, G, 4, NF / 2, GATED, OUT_FP8, SPLIT>(P, half, pool);
    half.strip += SF;
    half.strips = it.strips - SF;
    if (half.strips > 0) do_item<WEIGHT, G, 4, NF / 2, GATED, OUT_FP8, SPLIT>(P, half, pool);
  } else {
    do_item<WEIGHT, G, 4, NF, GATED, OUT_FP8, SPLIT>(P, it, pool);
  }
}

// The units [u0, u1) of a list of `tiles` x `units`. A unit is an output
// strip, or (fp8 out, where a row's 128 columns share a scale) 128 columns.
template <int WEIGHT, int G, bool GATED, bool OUT_FP8, bool SPLIT>
__device__ __forceinline__ void do_run(const GemmParams& P, int most, const uint32_t* pre,
                                       uint8_t* pool, int units, uint64_t u0, uint64_t u1) {
  constexpr int SF = GATED ? kFewFrags / 2 : kFewFrags;
  if (u0 >= u1) return;
  // division in 32 bits wherever the list allows it
  uint32_t tile = u1 >> 32 ? (uint32_t)(u0 / (uint32_t)units) : (uint32_t)u0 / (uint32_t)units;
  int unit = (int)(u0 - (uint64_t)tile * units);
  int e = expert_of_tile(pre, P.num_experts, tile);
  uint32_t end = (uint32_t)__builtin_amdgcn_readfirstlane((int)pre[e + 1]);
  for (uint64_t left = u1 - u0; left > 0;) {
    if (unit == units) {
      unit = 0;
      if (++tile == end) {
        e = expert_of_tile(pre, P.num_experts, tile);
        end = (uint32_t)__builtin_amdgcn_readfirstlane((int)pre[e + 1]);
      }
    }
    const int t = (int)(tile - (uint32_t)__builtin_amdgcn_readfirstlane((int)pre[e]));
    const int c = __builtin_amdgcn_readfirstlane((int)pre[P.num_experts + 1 + e]);
    Item it;
    it.e = e;
    const int first = few_first(c, most) + t * kFewRows;
    it.row0 = (int64_t)e * P.max_tokens + first;
    it.rows = c - first < kFewRows ? c - first : kFewRows;
    it.a = P.a + (uint64_t)it.row0 * P.k * (WEIGHT == kWeightFp8 ? 1 : 2);
    it.a_scales = WEIGHT == kWeightFp8 ? P.a_scales + (uint64_t)it.row0 * (P.k / 128) : nullptr;
    int here = units - unit;
    here = left < (uint64_t)here ? (int)left : here;
    int done = 1;
    it.strip = unit;
    if constexpr (OUT_FP8) {
      it.strip = unit * 8;
      it.strips = 8;
      do_item_rows<WEIGHT, G, kFewFrags, GATED, OUT_FP8, false>(P, it, pool);
    } else if constexpr (!SPLIT) {
      // as many strips as the workgroup holds, in items of like size
      const int items = (here + kFewWaves * SF - 1) / (kFewWaves * SF);
      it.strips = done = (here + items - 1) / items;
      do_item_rows<WEIGHT, G, kFewFrags, GATED, OUT_FP8, false>(P, it, pool);
    } else if (here >= SF) {
      it.strips = done = SF;
      do_item_rows<WEIGHT, G, kFewFrags, GATED, OUT_FP8, true>(P, it, pool);
    } else {
      // the run's last strips, fewer than a wavefront holds
      it.strips = 1;
      do_item_rows<WEIGHT, G, GATED ? 2 : 1, GATED, OUT_FP8, true>(P, it, pool);
    }
    unit += done;
    left -= done;
  }
}

// Workgroups: two a CU. A power of two, so that the runs need no division.
constexpr int kFewBlocksLog2 = 9;

template <int WEIGHT, int G, bool GATED, bool OUT_FP8>
__global__ void __launch_bounds__(kFewWaves * 64, 2) gemm_few_kernel(const GemmParams P, int most) {
  extern __shared__ __align__(16) uint8_t lds_raw[];
  __shared__ uint32_t scan[kFewWaves];
  __shared__ __align__(16) uint8_t pool[kPoolBytes];
  uint32_t* pre = reinterpret_cast<uint32_t*>(lds_raw);
  tile_prefix<kFewWaves * 64, true>(P, most, pre, scan);
  const uint32_t tiles = (uint32_t)__builtin_amdgcn_readfirstlane((int)pre[P.num_experts]);
  const int units = OUT_FP8 ? P.n / 128 : (P.n + 15) / 16;
  const uint64_t total = (uint64_t)tiles * units;
  // Workgroups are dealt to the XCDs in turn; neighbours in the list, which
  // share rows of A, go to one XCD and its L2.
  constexpr int LOG = kFewBlocksLog2;
  const uint32_t at = (blockIdx.x % kXcds << LOG) / kXcds + blockIdx.x / kXcds;
  const uint64_t u0 = total * at >> LOG, u1 = total * (at + 1) >> LOG;
  if (OUT_FP8 || total >> LOG >= kFewLong * (GATED ? kFewFrags / 2 : kFewFrags))
    do_run<WEIGHT, G, GATED, OUT_FP8, false>(P, most, pre, pool, units, u0, u1);
  else
    do_run<WEIGHT, G, GATED, OUT_FP8, true>(P, most, pre, pool, units, u0, u1);
}

template <int WEIGHT, int G, bool GATED, bool OUT_FP8>
hipError_t launch(const GemmParams& p, int most, hipStream_t stream) {
  gemm_few_kernel<WEIGHT, G, GATED, OUT_FP8>
      <<<1 << kFewBlocksLog2, kFewWaves * 64, tile_prefix_bytes(p.num_experts), stream>>>(p, most);
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
