// Low-rank adapters of many requests: kernel arguments, the workspace layout
// and the device helpers that the forward kernels (k_lora.hip) and the
// gradient's (k_lora_grad.hip) share.
#pragma once
#include "common.h"
#include "launch.h"
#include "rows.h"

namespace hm {

constexpr int kLoraUnit = 32;        // rows per unit: rows of one adapter that share its matrices' loads
constexpr int kLoraSlab = 512;       // output columns per block of the expanding kernels
constexpr int64_t kLoraMaxRows = 1 << 20;

// Rows of a call grouped by adapter: hdr[0] units of {adapter, first index
// into rows, count, 0}, the rows ascending within an adapter.
struct LoraRows {
  const int32_t* hdr;
  const int32_t* units;
  const int32_t* offsets;    // [L + 1] into rows
  const int32_t* rows;
  int64_t max_units;
};

struct LoraArgs {
  const uint16_t *x, *dy;    // bf16 [M][K], [M][N]
  const uint16_t *a, *b;     // bf16 [L][rank][K], [L][N][rank]
  const float* scales;
  const int32_t* ids;
  int64_t M, N, K;
  int rank, L;
  const uint16_t* base;      // [M][N] (forward), [M][K] (gradient) or null
  uint16_t* y;               // [M][N] (forward), [M][K] (gradient)
  float* h;                  // [M][rank]: written by the forward, read by the gradient
  float* part;               // fp32 [splits][M][rank] sums of the contracting kernels
  int splits;
  uint16_t *da, *db;
  LoraRows R;
};

// Byte offsets of the row grouping in the workspace; total a multiple of 256.
struct LoraWs {
  size_t hdr, units, counts, offsets, rows, cnt, part, total;
  int64_t max_units;
  int splits, splits_n;
};

inline int lora_rp(int rank) { return rank <= 16 ? 16 : (rank <= 32 ? 32 : (rank <= 64 ? 64 : 128)); }

hipError_t launch_lora_units(const int32_t* offsets, int L, int32_t* hdr, int32_t* units, hipStream_t st);
hipError_t launch_lora_shrink(const LoraArgs& g, hipStream_t st);
hipError_t launch_lora_expand(const LoraArgs& g, hipStream_t st);
hipError_t launch_lora_shrink_b(const LoraArgs& g, hipStream_t st);
hipError_t launch_lora_expand_a(const LoraArgs& g, hipStream_t st);
hipError_t launch_lora_outer(const LoraArgs& g, hipStream_t st);

#ifdef __HIPCC__
// fp32 -> two bf16 terms hi + lo: hi = bf16(v), lo = bf16(v - hi).  The sum
// carries v to 2^-16 of its size, far below the bf16 rounding of the results
// (2^-8), where hi alone would add an error as large as that rounding.
__device__ __forceinline__ void split8(const float v[8], u32x4_t* hi, u32x4_t* lo) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t h = pack_bf16(v[2 * j], v[2 * j + 1]);
    (*hi)[j] = h;
    (*lo)[j] = pack_bf16(v[2 * j] - lo_bf16(h), v[2 * j + 1] - hi_bf16(h));
  }
}

// 8 x 8 transpose of 16-bit values inside a lane: value i of out[j] is value
// j of in[i].
__device__ __forceinline__ void transpose8(const u32x4_t in[8], u32x4_t out[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int p = 0; p < 4; ++p)
      out[j][p] = __builtin_amdgcn_perm(in[2 * p + 1][j >> 1], in[2 * p][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
}

// Sum over the splits of row m's contracted values r0 .. r0 + 7, in split order.
__device__ __forceinline__ void load_h8(const float* __restrict__ part, int splits, int64_t M, int rank, int64_t m,
                                        int r0, float v[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (r0 >= rank) return;
  for (int s = 0; s < splits; ++s) {
    const float4* p = reinterpret_cast<const float4*>(part + ((int64_t)s * M + m) * rank + r0);
    const float4 a = p[0], b = p[1];
    v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
  }
}

// K steps (of 32) of the second product over [hi | lo] of RP rank columns,
// and the rank column lane quarter q supplies first in step s.  RP = 16: one
// step, quarters 0-1 hi, 2-3 lo.
template <int RP> struct RankSteps {
  static constexpr int S = RP == 16 ? 1 : RP / 16;
  __device__ static int r0(int s, int q) { return RP == 16 ? 8 * (q & 1) : 32 * (s % (RP / 32)) + 8 * q; }
  __device__ static bool lo(int s, int q) { return RP == 16 ? q >= 2 : s >= RP / 32; }
};

// MFMA operand (column = the lane's row m) of the second product.
template <int RP>
__device__ __forceinline__ void load_h_operand(const float* __restrict__ part, int splits, int64_t M, int rank, int64_t m,
                                               int q, u32x4_t hf[RankSteps<RP>::S]) {
  using RS = RankSteps<RP>;
  constexpr int half = RP == 16 ? 1 : RP / 32;
#pragma unroll
  for (int s = 0; s < half; ++s) {
    float v[8];
    load_h8(part, splits, M, rank, m, RS::r0(s, q), v);
    u32x4_t hi, lo;
    split8(v, &hi, &lo);
    if (RP == 16) {
      hf[0] = q >= 2 ? lo : hi;
    } else {
      hf[s] = hi;
      hf[half + s] = lo;
    }
  }
}

// Adds base to eight consecutive results and writes them (columns c .. c + 7
// of a row of n).
__device__ __forceinline__ void add_store8(const uint16_t* base, uint16_t* y, int64_t c, int64_t n, const float v[8]) {
  u32x4_t o = {0u, 0u, 0u, 0u};
  if (base) o = ld8_tail(base, c, n);
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = pack_bf16(lo_bf16(o[e]) + v[2 * e], hi_bf16(o[e]) + v[2 * e + 1]);
  st8_tail(y, c, n, o);
}

// Rows of [m0, m0 + kLoraUnit) without an adapter, columns [c0, c1): y = base
// (zeros without one).  One wave per row.
__device__ __forceinline__ void copy_rest(const LoraArgs& g, int64_t m0, int64_t n, int64_t c0, int64_t c1, bool zero_h) {
  const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
  for (int i = threadIdx.x >> 6; i < kLoraUnit; i += nw) {
    const int64_t m = m0 + i;
    if (m >= g.M) break;
    const int e = g.ids[m];
    if (e >= 0 && e < g.L) continue;
    if (g.base != g.y)
      for (int64_t c = c0 + 8 * lane; c < c1; c += 512)
        st8_tail(g.y + m * n, c, n, g.base ? ld8_tail(g.base + m * n, c, n) : (u32x4_t){0u, 0u, 0u, 0u});
    if (zero_h)
      for (int r = lane; r < g.rank; r += 64) g.h[m * g.rank + r] = 0.f;
  }
}
#endif

}  // namespace hm
