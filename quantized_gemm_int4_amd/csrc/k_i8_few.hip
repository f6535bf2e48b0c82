// Products of 8-bit integer layers for few rows (up to 1024): bound by reading the
// weights, once where the rows are one group (up to 128), from L2 for the other groups.
//
// A block has 16 NB weight rows, NB = 1 .. 4 (pairs: NB = 2 or 4, half of them gate rows and half the up rows that
// belong to them) against a group of up to 128 rows of x, and its four waves split the contraction:
// wave w takes the steps w, w + 4, ... of 128 bytes of every row, each by itself, so that
// the block reads its rows from end to end.  Direct buffer-to-LDS copies bring them
// in, eight lanes a line, and the operands of the 16x16x64 MFMA (lane L: row L % 16, 16
// bytes at 16 (L / 16) of 64) are read from there.  Loaded straight into the
// operand, a wave's 16 lanes each ask for a line of their own, and a compute unit takes
// 37 bytes a nanosecond, from L2 too (m = 64, n = 1958, k = 6784 17.7 us, now 11.6; m = 48, n = 28672, k = 4096
// 36.5, 29.9; gated m = 54, n = 1810, k = 4608 13.8, 7.6).  Rows past the last are range-checked away and
// cost no traffic.  The waves' exact integer sums meet in LDS.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "common.h"
#include "i8.h"
#include "i8_tile.h"

namespace hm {

namespace {

constexpr int kBlock = 2048;                       // 16 rows x 128 bytes
constexpr int W = 4;                               // waves

__device__ __forceinline__ i32x4_t mma16(u32x4_t a, u32x4_t b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
}

// MB: 16-row blocks of x, NB: 16-row blocks of weights (pairs: gate and up), S: steps on their way.
// LDS of a wave: its steps, then its sums
template <int MB, int NB, int S> constexpr int kFewOwn = S * (NB + MB) * kBlock > NB * MB * 1024 ? S * (NB + MB) * kBlock : NB * MB * 1024;

template <int MB, int NB, int S, int EPI>
__global__ void __launch_bounds__(64 * W)
k_i8_few(TileArgs a, uint32_t total, int groups, int per) {
  extern __shared__ __align__(1024) uint8_t lds[];
  constexpr int kStage = (NB + MB) * kBlock, kOwn = kFewOwn<MB, NB, S>, kCopies = 2 * (NB + MB);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t K = a.kbytes;
  constexpr int kOut = kPairs<EPI> ? NB / 2 : NB, kCols = 16 * kOut;    // 16-column blocks, columns of the output
  // the groups of rows after each other on an XCD, whose L2 then has the weights
  const uint32_t t0 = number_of(total, blockIdx.x, gridDim.x, 0);
  if (t0 >= total) return;
  const uint32_t tc = t0 / (uint32_t)groups;
  const int64_t c0 = (int64_t)tc * kCols, r0 = (int64_t)(t0 - tc * groups) * per;
  const int rows = (int)min((int64_t)per, a.rows - r0);
  uint8_t* const own = lds + wave * kOwn;
  // a step: 128 bytes of every row; the wave's are W apart
  const uint8_t* pw = a.p + c0 * K + wave * 128;
  const uint8_t* px = a.q + r0 * K + wave * 128;
  int64_t lw = a.p_bytes - c0 * K - wave * 128, lx = rows * K - wave * 128;
  const uint32_t ld = (uint32_t)K;
  // copy i of a block: rows 8 i + lane / 8, chunk c of 16 bytes at place c ^ ((row >> 1) & 7)
  uint32_t vo[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) vo[i] = (uint32_t)(8 * i + (lane >> 3)) * ld + 16 * ((lane & 7) ^ ((lane >> 4) | (4 * i)));
  int left = (int)(K / 128) - wave;                // steps from the next one to copy
  auto fetch = [&](uint8_t* stage) __attribute__((always_inline)) {
    const bool any = left > 0;                     // past the end: zeros, so that the waits can count
    const rsrc_t rw = make_rsrc(pw, any && lw > 0 ? (uint64_t)lw : 0), rx = make_rsrc(px, any ? (uint64_t)lx : 0);
    const rsrc_t ru = kPairs<EPI> ? make_rsrc(pw + a.p_bytes, any && lw > 0 ? (uint64_t)lw : 0) : rw;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        b2lds16(b < kOut ? rw : ru, vo[i] + (uint32_t)(b % kOut) * 16 * ld, 0u, stage + b * kBlock + i * 1024);
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) b2lds16(rx, vo[i] + (uint32_t)b * 16 * ld, 0u, stage + (NB + b) * kBlock + i * 1024);
    pw += 128 * W;
    px += 128 * W;
    lw -= 128 * W;
    lx -= 128 * W;
    left -= W;
  };
  int steps = ((int)(K / 128) - wave + W - 1) / W;
#pragma unroll
  for (int s = 0; s < S; ++s) fetch(own + s * kStage);
  // operand of part ks (64 bytes): row lane % 16, chunk 4 ks + lane / 16
  uint32_t at[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
    at[ks] = (uint32_t)(uintptr_t)(lds_void_t*)own + (lane & 15) * 128 + 16 * ((4 * ks + (lane >> 4)) ^ ((lane >> 1) & 7));

  i32x4_t acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = (i32x4_t){0, 0, 0, 0};
  int st = 0;
  for (; steps > 0; --steps) {
    __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 1) * kCopies) : "memory");
    u32x4_t wv[NB][2], xv[MB][2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
      for (int b = 0; b < NB; ++b) wv[b][ks] = *(const lds_u32x4_t*)(at[ks] + st * kStage + b * kBlock);
#pragma unroll
      for (int b = 0; b < MB; ++b) xv[b][ks] = *(const lds_u32x4_t*)(at[ks] + st * kStage + (NB + b) * kBlock);
    }
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");             // the stage is in registers
    fetch(own + st * kStage);
    st = st + 1 == S ? 0 : st + 1;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = mma16(wv[i][ks], xv[j][ks], acc[i][j]);
  }
  // the wave's sums take the place of its steps
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  auto sums = [&](int w, int i, int j, int l) -> i32x4_t& { return reinterpret_cast<i32x4_t*>(lds + w * kOwn)[(i * MB + j) * 64 + l]; };
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) sums(wave, i, j, lane) = acc[i][j];
  __syncthreads();
  // lane of a block: row of x l16, weight rows 4 part .. + 3
  for (int t = tid; t < kOut * MB * 64; t += 64 * W) {
    const int i = t / (MB * 64), j = (t / 64) % MB, l = t & 63;
    const int64_t m = r0 + 16 * j + (l & 15), n = c0 + 16 * i + 4 * (l >> 4);
    if (m >= r0 + rows || n >= a.cols) continue;
    i32x4_t s[kPairs<EPI> ? 2 : 1];
#pragma unroll
    for (int h = 0; h < (kPairs<EPI> ? 2 : 1); ++h) {
      s[h] = sums(0, i + h * kOut, j, l);
#pragma unroll
      for (int v = 1; v < W; ++v) s[h] += sums(v, i + h * kOut, j, l);
    }
    const float sq = a.qs[m];
    constexpr int kOuts = EPI == EPI_GATED_GRAD ? 2 : 1;
    float f[kOuts][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t c = min(n + e, a.cols - 1);
      f[0][e] = (float)s[0][e] * sq * a.ps[c];
      if constexpr (kPairs<EPI>) {
        const float g = f[0][e], u = (float)s[1][e] * sq * a.ps[a.cols + c];
        if constexpr (EPI == EPI_GATED) f[0][e] = gated(g, u);
        else gated_grad(g, u, bf16_to_f32(a.dh[m * a.cols + c]), f[0][e], f[1][e]);
      }
    }
#pragma unroll
    for (int k = 0; k < kOuts; ++k) {
      uint16_t* y = a.out + (m * kOuts + k) * a.cols + n;
      const uint32_t lo = pack_bf16(f[k][0], f[k][1]), hi = pack_bf16(f[k][2], f[k][3]);
      if (n + 3 < a.cols) {
        *reinterpret_cast<u32x2_a2_t*>(y) = (u32x2_t){lo, hi};
      } else {
        const uint64_t v = lo | ((uint64_t)hi << 32);
        for (int e = 0; n + e < a.cols; ++e) y[e] = (uint16_t)(v >> (16 * e));
      }
    }
  }
}

template <int MB, int NB, int S, int EPI>
hipError_t go(const TileArgs& a, const FewPlan& p, hipStream_t st) {
  constexpr int kCols = 16 * (kPairs<EPI> ? NB / 2 : NB), kLds = W * kFewOwn<MB, NB, S>;
  auto kern = &k_i8_few<MB, NB, S, EPI>;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (attr != hipSuccess) return attr;
  const uint32_t total = (uint32_t)((a.cols + kCols - 1) / kCols * p.groups);
  hipLaunchKernelGGL(kern, dim3(8 * ((total + 7) / 8)), dim3(64 * W), kLds, st, a, total, p.groups, p.rows);
  return hipGetLastError();
}

// Two steps on their way where every compute unit has one block at most and LDS the room, one where several share it
// (m = 64, n = 14336, k = 4096, 224 blocks: 17.8 us with two, 19.5 with one; m = 48, n = 28672, 448 blocks: 32.7, 29.9).
template <int MB, int NB, int EPI>
hipError_t steps(const TileArgs& a, const FewPlan& p, hipStream_t st) {
  constexpr int kCols = 16 * (kPairs<EPI> ? NB / 2 : NB);
  if constexpr (2 * W * (NB + MB) * kBlock <= 160 * 1024) {
    if (a.cols <= 256 / p.groups * kCols) return go<MB, NB, 2, EPI>(a, p, st);
  }
  return go<MB, NB, 1, EPI>(a, p, st);
}

template <int MB, int EPI>
hipError_t blocks(const TileArgs& a, const FewPlan& p, hipStream_t st) {
  constexpr int kMost = i8_few_most(MB, kPairs<EPI>);
  if constexpr (!kPairs<EPI>) {
    if (p.nb == 1) return steps<MB, 1, EPI>(a, p, st);
    if constexpr (kMost >= 3) {
      if (p.nb == 3) return steps<MB, 3, EPI>(a, p, st);
    }
  }
  if constexpr (kMost >= 4) {
    if (p.nb == 4) return steps<MB, 4, EPI>(a, p, st);
  }
  return steps<MB, 2, EPI>(a, p, st);
}

template <int EPI>
hipError_t rows(const TileArgs& a, const FewPlan& p, hipStream_t st) {
  switch (p.rows / 16) {
    case 1: return blocks<1, EPI>(a, p, st);
    case 2: return blocks<2, EPI>(a, p, st);
    case 3: return blocks<3, EPI>(a, p, st);
    case 4: return blocks<4, EPI>(a, p, st);
    case 5: case 6: return blocks<6, EPI>(a, p, st);
    default: return blocks<8, EPI>(a, p, st);
  }
}

}  // namespace

hipError_t launch_i8_few(const TileArgs& a, const FewPlan& p, int kind, hipStream_t st) {
  switch (kind) {
    case I8_FORWARD: return rows<EPI_SCALE>(a, p, st);
    case I8_GATED: return rows<EPI_GATED>(a, p, st);
    default: return rows<EPI_GATED_GRAD>(a, p, st);
  }
}

}  // namespace hm
