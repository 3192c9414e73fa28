// Root-mean-square norm of x plus the residual, with the new residual and an
// output in bf16 or in e4m3 with a scale per 128 columns.
//
// Mathematics, for one row in fp32: h = x + residual; residual_out = h
// rounded to bf16; y = h / sqrt(mean(h^2) + eps) * weight, taken from h
// before that rounding; out = y in bf16, or codes e4m3(y * (448 / amax)) and
// scales amax / 448 of each 128 columns, as the fp8 dispatch quantizes (tiny
// blocks apart: block_scale).
//
// Design: one workgroup a row (one wavefront for short rows, four rows a
// workgroup), the row in registers from its one read to its one write: the
// bytes moved are the floor's. A thread holds chunks of 8 columns, so 16
// lanes hold the 128 columns that share a scale and reduce amax in four
// steps. Bound: HBM for many rows (16384 x 7168 to fp8 143 us, 5.8 TB/s, where a
// copy reaches 5.96), latency for few (one row 3.1 us, 128 of fp32 3.8).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_gemm.h"
#include "norm.h"

namespace llmoe {
namespace {

__device__ __forceinline__ void unpack8(const v4u v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ v4u pack8(const float (&f)[8]) {
  return v4u{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]),
             bf16_pair(f[6], f[7])};
}

constexpr int kFewTokens = 256;

// ROW: threads of a row; C: chunks of 8 columns a thread holds. A workgroup
// of max(ROW, 256) threads takes rows side by side.
template <int ROW, int C, bool X_FP32, bool RESIDUAL, bool OUT_FP8>
__global__ void __launch_bounds__(ROW < 256 ? 256 : ROW) norm_kernel(const NormParams P) {
  constexpr int BLOCK = ROW < 256 ? 256 : ROW;
  __shared__ float part[BLOCK / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int t0 = tid % ROW;
  const int64_t row = (int64_t)blockIdx.x * (BLOCK / ROW) + tid / ROW;
  const bool live = row < P.num_tokens;
  const int chunks = P.hidden / 8;
  const uint64_t base = (uint64_t)(live ? row : 0) * chunks;
  // every load goes out before any is used; those behind the row read its
  // last chunk again, and count as zeros
  v4u xr[C][X_FP32 ? 2 : 1], rr[C], wt[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = t0 + c * ROW < chunks ? t0 + c * ROW : chunks - 1;
    if constexpr (X_FP32) {
      const v4u* x = reinterpret_cast<const v4u*>(P.x) + 2 * (base + i);
      xr[c][0] = x[0];
      xr[c][1] = x[1];
    } else {
      xr[c][0] = reinterpret_cast<const v4u*>(P.x)[base + i];
    }
    rr[c] = RESIDUAL ? reinterpret_cast<const v4u*>(P.residual)[base + i] : v4u{0, 0, 0, 0};
    wt[c] = reinterpret_cast<const v4u*>(P.weight)[i];
  }
  float h[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const bool in = t0 + c * ROW < chunks;
    if constexpr (X_FP32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[c][j] = __uint_as_float(xr[c][0][j]);
        h[c][4 + j] = __uint_as_float(xr[c][1][j]);
      }
    } else {
      unpack8(xr[c][0], h[c]);
    }
    if constexpr (RESIDUAL) {
      float r[8];
      unpack8(rr[c], r);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] += r[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) h[c][j] = in ? h[c][j] : 0.0f;
  }
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(h[c][j], h[c][j], sum);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
  if constexpr (ROW > 64) {
    if (lane == 0) part[tid / 64] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < ROW / 64; ++w) sum += part[w];
  }
  const float scale = 1.0f / sqrtf(sum / (float)P.hidden + P.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = t0 + c * ROW;
    const bool in = live && i < chunks;
    if (P.residual_out && in) reinterpret_cast<v4u*>(P.residual_out)[base + i] = pack8(h[c]);
    float w[8], y[8];
    unpack8(wt[c], w);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = h[c][j] * scale * w[j];
    if constexpr (OUT_FP8) {
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y[j]));  // NaN is ignored
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) amax = fmaxf(amax, __shfl_xor(amax, d, 64));
      const auto [unit, inv] = block_scale(amax);
      if (in) {
        reinterpret_cast<uint2*>(P.out)[base + i] =
            make_uint2(e4m3_pack4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                       e4m3_pack4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
        if ((i & 15) == 0) P.out_scales[(base + i) / 16] = unit;
      }
    } else if (in) {
      reinterpret_cast<v4u*>(P.out)[base + i] = pack8(y);
    }
  }
}

// The norm of `rows` rows from row `first` on.
NormParams rows_from(const NormParams& p, uint64_t first, int rows) {
  NormParams q = p;
  const uint64_t at = first * p.hidden;
  q.x += at * (p.x_fp32 ? 4 : 2);
  if (q.residual) q.residual += at * 2;
  if (q.residual_out) q.residual_out += at * 2;
  q.out += at * (p.out_fp8 ? 1 : 2);
  if (p.out_fp8) q.out_scales += at / 128;
  q.num_tokens = rows;
  return q;
}

template <int ROW, int C, bool X_FP32, bool RESIDUAL>
hipError_t launch(const NormParams& p, hipStream_t stream) {
  constexpr int BLOCK = ROW < 256 ? 256 : ROW, ROWS = BLOCK / ROW;
  // A grid has fewer than 2^32 threads (one of more is cut off without an
  // error): 2^31 threads a launch, 2^21 rows of 1024 threads at the least.
  constexpr int kMost = (int)((1ll << 31) / ROW);
  for (int64_t first = 0; first < p.num_tokens; first += kMost) {
    const int64_t left = p.num_tokens - first;
    const NormParams q = rows_from(p, (uint64_t)first, (int)(left < kMost ? left : kMost));
    const unsigned blocks = ((unsigned)q.num_tokens + ROWS - 1) / ROWS;
    if (q.out_fp8) norm_kernel<ROW, C, X_FP32, RESIDUAL, true><<<blocks, BLOCK, 0, stream>>>(q);
    else norm_kernel<ROW, C, X_FP32, RESIDUAL, false><<<blocks, BLOCK, 0, stream>>>(q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool X_FP32, bool RESIDUAL>
hipError_t launch_x(const NormParams& p, hipStream_t stream) {
  const int chunks = p.hidden / 8;
  if (chunks <= 64) return launch<64, 1, X_FP32, RESIDUAL>(p, stream);
  if (chunks <= 128) return launch<64, 2, X_FP32, RESIDUAL>(p, stream);
  if (chunks <= 256) return launch<256, 1, X_FP32, RESIDUAL>(p, stream);
  // Few rows leave the GPU idle: more threads a row, fewer chunks a thread.
  if (p.num_tokens <= kFewTokens && chunks <= 1024)
    return chunks <= 512 ? launch<512, 1, X_FP32, RESIDUAL>(p, stream)
                         : launch<1024, 1, X_FP32, RESIDUAL>(p, stream);
  if (chunks <= 512) return launch<256, 2, X_FP32, RESIDUAL>(p, stream);
  if (chunks <= 1024) return launch<256, 4, X_FP32, RESIDUAL>(p, stream);
  if (chunks <= 2048) return launch<512, 4, X_FP32, RESIDUAL>(p, stream);
  return launch<1024, 4, X_FP32, RESIDUAL>(p, stream);
}

}  // namespace

hipError_t launch_norm(const NormParams& p, hipStream_t stream) {
  if (p.num_tokens == 0) return hipSuccess;
  if (p.residual)
    return p.x_fp32 ? launch_x<true, true>(p, stream) : launch_x<false, true>(p, stream);
  return p.x_fp32 ? launch_x<true, false>(p, stream) : launch_x<false, false>(p, stream);
}

}  // namespace llmoe
