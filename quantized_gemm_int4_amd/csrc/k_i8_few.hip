// Products of 8-bit integer layers for few rows (decoding: up to 64): bound by
// reading the weights once.
//
// A block has 16 NB weight rows (pairs: 16 gate rows and the 16 up rows that
// belong to them) against all rows of x, and its waves split the contraction:
// wave w takes the pieces w, w + waves, ... of 256 bytes of every row, so that the
// block reads its rows from end to end.  Weights go straight from global memory
// into the operand of the 16x16x64 MFMA (lane L: row L % 16, 16 bytes at 16 (L / 16) of
// 64), rows of x into the other; rows past the last are range-checked away and
// cost no traffic.  The waves' exact integer sums meet in LDS.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "common.h"
#include "i8.h"
#include "i8_tile.h"

namespace hm {

namespace {

constexpr int kPiece = 256;                        // bytes of a row that a wave takes at a time

__device__ __forceinline__ i32x4_t mma16(u32x4_t a, u32x4_t b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
}

__device__ __forceinline__ u32x4_t load16(rsrc_t r, uint32_t at) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}

// MB: 16-row blocks of x, NB: 16-row blocks of weights a wave (pairs: gate and up), W: waves of a block.
template <int MB, int NB, int W, int EPI>
__global__ void __launch_bounds__(64 * W)
k_i8_few(TileArgs a) {
  extern __shared__ __align__(16) i32x4_t sums[];  // [W][NB * MB][64]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, part = lane >> 4;
  const int64_t K = a.kbytes;
  constexpr int kOut = kPairs<EPI> ? NB / 2 : NB, kCols = 16 * kOut;    // 16-column blocks, columns of the output
  const int64_t c0 = (int64_t)blockIdx.x * kCols;
  const uint8_t* w[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    // rows behind the last repeat it; their columns are not stored
    const int64_t n = min(c0 + 16 * (b % kOut) + l16, a.cols - 1);
    w[b] = a.p + (n + b / kOut * a.cols) * K + 16 * part;
  }
  const rsrc_t rx = make_rsrc(a.q, (uint64_t)a.rows * (uint64_t)K);
  uint32_t x[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) x[b] = (uint32_t)(16 * b + l16) * (uint32_t)K + 16 * part;

  i32x4_t acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = (i32x4_t){0, 0, 0, 0};
  auto run = [&](int64_t k, auto count) __attribute__((always_inline)) {
    constexpr int U = count.value;                 // 64-byte parts
    u32x4_t wv[NB][U], xv[MB][U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < NB; ++b) wv[b][u] = ld16(w[b] + k + 64 * u);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < MB; ++b) xv[b][u] = load16(rx, x[b] + (uint32_t)k + 64 * u);
    __builtin_amdgcn_sched_barrier(0);             // all of a piece's loads are in flight before the first is waited for
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = mma16(wv[i][u], xv[j][u], acc[i][j]);
  };
  const int64_t whole = K / kPiece * kPiece;
  for (int64_t k = (int64_t)wave * kPiece; k < whole; k += W * kPiece) run(k, std::integral_constant<int, 4>());
  // the last 128 bytes of an odd multiple: the wave whose turn it is
  if (K > whole && (whole / kPiece) % W == wave) run(whole, std::integral_constant<int, 2>());

#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) sums[(wave * NB * MB + i * MB + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // lane of a block: row of x l16, weight rows 4 part .. + 3
  for (int t = tid; t < kOut * MB * 64; t += 64 * W) {
    const int i = t / (MB * 64), j = (t / 64) % MB, l = t & 63;
    const int64_t m = 16 * j + (l & 15), n = c0 + 16 * i + 4 * (l >> 4);
    if (m >= a.rows || n >= a.cols) continue;
    i32x4_t s[kPairs<EPI> ? 2 : 1];
#pragma unroll
    for (int h = 0; h < (kPairs<EPI> ? 2 : 1); ++h) {
      s[h] = sums[((i + h * kOut) * MB + j) * 64 + l];
#pragma unroll
      for (int v = 1; v < W; ++v) s[h] += sums[(v * NB * MB + (i + h * kOut) * MB + j) * 64 + l];
    }
    const float sq = a.qs[m];
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t c = min(n + e, a.cols - 1);
      f[e] = (float)s[0][e] * sq * a.ps[c];
      if constexpr (kPairs<EPI>) f[e] = silu_f(f[e]) * ((float)s[1][e] * sq * a.ps[a.cols + c]);
    }
    uint16_t* y = a.out + m * a.cols + n;
    const uint32_t lo = pack_bf16(f[0], f[1]), hi = pack_bf16(f[2], f[3]);
    if (n + 3 < a.cols) {
      *reinterpret_cast<u32x2_a2_t*>(y) = (u32x2_t){lo, hi};
    } else {
      const uint64_t v = lo | ((uint64_t)hi << 32);
      for (int e = 0; n + e < a.cols; ++e) y[e] = (uint16_t)(v >> (16 * e));
    }
  }
}

template <int MB, int NB, int W, int EPI>
hipError_t go(const TileArgs& a, hipStream_t st) {
  constexpr int kCols = 16 * (kPairs<EPI> ? NB / 2 : NB), kLds = W * NB * MB * 1024;
  auto kern = &k_i8_few<MB, NB, W, EPI>;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(kern, dim3((unsigned)((a.cols + kCols - 1) / kCols)), dim3(64 * W), kLds, st, a);
  return hipGetLastError();
}

// Waves: eight for one block of rows, four for more, whose loads fill as much (n = 28672, k = 4096, four weight
// blocks: m = 1 21.2 us with either, m = 48 29.2 against 32.4; n = 14336: m = 1 11.3 with eight, 12.4 with four).
template <int MB, int EPI>
hipError_t blocks(const TileArgs& a, hipStream_t st) {
  constexpr int W = MB == 1 ? 8 : 4;
  switch (i8_few_blocks(a.cols, kPairs<EPI>)) {
    case 4: return go<MB, 4, W, EPI>(a, st);
    case 2: return go<MB, 2, W, EPI>(a, st);
    default:
      if constexpr (!kPairs<EPI>) return go<MB, 1, W, EPI>(a, st);
      return hipErrorInvalidValue;
  }
}

template <int EPI>
hipError_t rows(const TileArgs& a, hipStream_t st) {
  switch ((a.rows + 15) / 16) {
    case 1: return blocks<1, EPI>(a, st);
    case 2: return blocks<2, EPI>(a, st);
    case 3: return blocks<3, EPI>(a, st);
    default: return blocks<4, EPI>(a, st);
  }
}

}  // namespace

hipError_t launch_i8_few(const TileArgs& a, int kind, hipStream_t st) {
  return kind == I8_GATED ? rows<EPI_GATED>(a, st) : rows<EPI_SCALE>(a, st);
}

}  // namespace hm
