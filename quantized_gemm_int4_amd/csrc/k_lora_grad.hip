// Gradient of the low-rank adapters.  For the rows m of adapter e:
//   g[m] = s_e B_e^T dy[m]                    contraction over N
//   dx[m] = dx_base[m] + A_e^T g[m]           contraction over the rank
//   da_e = sum_m g[m] x[m]^T,  db_e = sum_m dy[m] h[m]^T    over the rows
// Every product runs on the bf16 MFMA, whose operands want eight consecutive
// values of the contracted axis per lane.  Where that axis is the strided one
// in memory (the rank of A, the columns of B, the rows of x and dy) a lane
// loads eight rows of a few neighbouring columns and transposes them in its
// registers; each of those columns is one MFMA's.
#include "lora.h"

namespace hm {

// Values c .. c + W - 1 (W = 1, 2, 4, 8) of eight rows, transposed: value i
// of out[j] is column c + j of row i (0 for rows not in `ok`).
template <int W>
__device__ __forceinline__ void load_cols8(const uint16_t* p, int64_t stride, int ok, u32x4_t out[W]) {
  if constexpr (W == 8) {
    u32x4_t in[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) in[i] = i < ok ? ld16(p + i * stride) : (u32x4_t){0u, 0u, 0u, 0u};
    transpose8(in, out);
  } else {
    uint32_t in[8][(W + 1) / 2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (W == 4) {
        const u32x2_t v = i < ok ? *reinterpret_cast<const u32x2_t*>(p + i * stride) : (u32x2_t){0u, 0u};
        in[i][0] = v[0];
        in[i][1] = v[1];
      } else if constexpr (W == 2) {
        in[i][0] = i < ok ? *reinterpret_cast<const uint32_t*>(p + i * stride) : 0u;
      } else {
        in[i][0] = i < ok ? p[i * stride] : 0u;
      }
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        out[j][k] = __builtin_amdgcn_perm(in[2 * k + 1][j >> 1], in[2 * k][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
  }
}

// grid (splits, units): g = s_e B_e^T dy, the contraction over N split as
// k_lora_shrink splits K.  Lane (c, q) supplies rank columns W c + j of B.
template <int RP>
__global__ void __launch_bounds__(256) k_lora_shrink_b(LoraArgs g) {
  constexpr int W = RP / 16, LD = RP + 4;
  __shared__ float red[4][kLoraUnit][LD];
  const int u = blockIdx.y;
  if (u >= g.R.hdr[0]) return;
  const int32_t* un = g.R.units + 4 * (int64_t)u;
  const int e = un[0], first = un[1], count = un[2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const int64_t steps = (g.N + 31) / 32, waves = 4 * (int64_t)g.splits, wi = (int64_t)blockIdx.x * 4 + wave;
  const int64_t s0 = steps * wi / waves, s1 = steps * (wi + 1) / waves;
  const uint16_t* dp[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) dp[t] = g.dy + (int64_t)g.R.rows[first + min(16 * t + c, count - 1)] * g.N;
  const uint16_t* bp = g.b + (int64_t)e * g.N * g.rank + W * c;
  const bool in_rank = W * c < g.rank;
  f32x4_t acc[2][W];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < W; ++j) acc[t][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  for (int64_t s = s0; s < s1; ++s) {
    const int64_t n = 32 * s + 8 * q;
    u32x4_t dv[2], bv[W];
#pragma unroll
    for (int t = 0; t < 2; ++t) dv[t] = n < g.N ? ld8_tail(dp[t], n, g.N) : (u32x4_t){0u, 0u, 0u, 0u};
    const int64_t left = g.N - n;
    load_cols8<W>(bp + n * g.rank, g.rank, in_rank ? (int)(left < 8 ? left : 8) : 0, bv);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int t = 0; t < 2; ++t) acc[t][j] = mfma_bf16(bv[j], dv[t], acc[t][j]);
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int j = 0; j < W; ++j) red[wave][16 * t + c][W * (4 * q + v) + j] = acc[t][j][v];
  __syncthreads();
  const float sc = g.scales[e];
  float* out = g.part + (int64_t)blockIdx.x * g.M * g.rank;
  for (int i = threadIdx.x; i < count * RP; i += 256) {
    const int row = i / RP, r = i % RP;
    if (r < g.rank)
      out[(int64_t)g.R.rows[first + row] * g.rank + r] =
          sc * ((red[0][row][r] + red[1][row][r]) + (red[2][row][r] + red[3][row][r]));
  }
}

// grid (column slabs of K, units + groups of rows without an adapter): dx =
// dx_base + A_e^T g.  A wave's 128 columns: lane (c, q) supplies column k0 +
// 8 c + j to MFMA j and ends up with columns k0 + 8 (4 q + v) + j of row c.
template <int RP>
__global__ void __launch_bounds__(256) k_lora_expand_a(LoraArgs g) {
  using RS = RankSteps<RP>;
  constexpr int half = RP == 16 ? 1 : RP / 32;
  const int64_t c0 = (int64_t)blockIdx.x * kLoraSlab, c1 = min(c0 + kLoraSlab, g.K);
  if (blockIdx.y >= g.R.max_units) {
    copy_rest(g, (blockIdx.y - g.R.max_units) * kLoraUnit, g.K, c0, c1, false);
    return;
  }
  const int u = blockIdx.y;
  if (u >= g.R.hdr[0]) return;
  const int32_t* un = g.R.units + 4 * (int64_t)u;
  const int e = un[0], first = un[1], count = un[2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  int64_t m[2];
  u32x4_t gf[2][RS::S];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    m[t] = g.R.rows[first + min(16 * t + c, count - 1)];
    load_h_operand<RP>(g.part, g.splits, g.M, g.rank, m[t], q, gf[t]);
  }
  const uint16_t* A = g.a + (int64_t)e * g.rank * g.K;
  for (int64_t k0 = c0 + 128 * wave; k0 < c1; k0 += 512) {
    f32x4_t acc[2][8];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[t][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < half; ++s) {
      const int r0 = RS::r0(s, q);
      u32x4_t av[8];
      load_cols8<8>(A + (int64_t)r0 * g.K + k0 + 8 * c, g.K, r0 < g.rank ? 8 : 0, av);
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          acc[t][j] = mfma_bf16(av[j], gf[t][s], acc[t][j]);
          if (RP != 16) acc[t][j] = mfma_bf16(av[j], gf[t][half + s], acc[t][j]);
        }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (16 * t + c >= count) continue;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float o[8] = {acc[t][0][v], acc[t][1][v], acc[t][2][v], acc[t][3][v],
                            acc[t][4][v], acc[t][5][v], acc[t][6][v], acc[t][7][v]};
        add_store8(g.base ? g.base + m[t] * g.K : nullptr, g.y + m[t] * g.K, k0 + 32 * q + 8 * v, g.K, o);
      }
    }
  }
}

// grid (128-column tiles, rank chunks of 16 RB, adapters): the contraction
// over an adapter's rows.  COLS rows of z (x or dy) of `n` columns against f
// (g summed over its splits, or h): out[r][col] (da) or out[col][r] (db).
// The block's waves split the rows; their sums meet in LDS, in wave order.
template <int RB, bool DB>
__global__ void __launch_bounds__(256) k_lora_outer(LoraArgs g) {
  constexpr int RC = 16 * RB;
  __shared__ float red[RC][132];
  const int e = blockIdx.z, r00 = blockIdx.y * RC;
  const int64_t n = DB ? g.N : g.K, k0 = 128 * (int64_t)blockIdx.x;
  const uint16_t* z = DB ? g.dy : g.x;
  const float* f = DB ? g.h : g.part;
  const int splits = DB ? 1 : g.splits;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const int beg = g.M ? g.R.offsets[e] : 0, end = g.M ? g.R.offsets[e + 1] : 0;
  const int64_t col = k0 + 8 * c;
  f32x4_t acc[8][RB];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < RB; ++i) acc[j][i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  for (int b = beg + 32 * wave; b < end; b += 128) {
    u32x4_t in[8], zv[8], hi[RB], lo[RB];
    float fv[RB][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool ok = b + 8 * q + i < end;
      const int64_t m = ok ? g.R.rows[b + 8 * q + i] : 0;
      in[i] = ok && col < n ? ld8_tail(z + m * n, col, n) : (u32x4_t){0u, 0u, 0u, 0u};
#pragma unroll
      for (int k = 0; k < RB; ++k) {
        const int r = r00 + 16 * k + c;
        float v = 0.f;
        if (ok && r < g.rank)
          for (int s = 0; s < splits; ++s) v += f[((int64_t)s * g.M + m) * g.rank + r];
        fv[k][i] = v;
      }
    }
    transpose8(in, zv);
#pragma unroll
    for (int k = 0; k < RB; ++k) split8(fv[k], &hi[k], &lo[k]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int k = 0; k < RB; ++k) {
        if (DB) {
          acc[j][k] = mfma_bf16(hi[k], zv[j], acc[j][k]);
          acc[j][k] = mfma_bf16(lo[k], zv[j], acc[j][k]);
        } else {
          acc[j][k] = mfma_bf16(zv[j], hi[k], acc[j][k]);
          acc[j][k] = mfma_bf16(zv[j], lo[k], acc[j][k]);
        }
      }
  }
  // DB: lane holds columns 8 c + j, rank 16 k + 4 q + v; else rank 16 k + c, columns 8 (4 q + v) + j
  for (int w = 0; w < 4; ++w) {
    if (w == wave)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int k = 0; k < RB; ++k)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            float* p = DB ? &red[16 * k + 4 * q + v][8 * c + j] : &red[16 * k + c][8 * (4 * q + v) + j];
            *p = w == 0 ? acc[j][k][v] : *p + acc[j][k][v];
          }
    __syncthreads();
  }
  if (DB) {
    for (int i = threadIdx.x; i < 128 * RC / 8; i += 256) {
      const int cc = i / (RC / 8), r = 8 * (i % (RC / 8));
      if (k0 + cc >= n || r00 + r >= g.rank) continue;
      u32x4_t o;
#pragma unroll
      for (int p = 0; p < 4; ++p) o[p] = pack_bf16(red[r + 2 * p][cc], red[r + 2 * p + 1][cc]);
      st16(g.db + ((int64_t)e * n + k0 + cc) * g.rank + r00 + r, o);
    }
  } else {
    for (int i = threadIdx.x; i < 16 * RC; i += 256) {
      const int r = i / 16, cc = 8 * (i % 16);
      if (r00 + r >= g.rank) continue;
      u32x4_t o;
#pragma unroll
      for (int p = 0; p < 4; ++p) o[p] = pack_bf16(red[r][cc + 2 * p], red[r][cc + 2 * p + 1]);
      st16(g.da + ((int64_t)e * g.rank + r00 + r) * n + k0 + cc, o);
    }
  }
}

#define HM_LORA_RANKS(K, grid)                                                        \
  switch (lora_rp(g.rank)) {                                                          \
    case 16: hipLaunchKernelGGL(K<16>, grid, dim3(256), 0, st, g); break;             \
    case 32: hipLaunchKernelGGL(K<32>, grid, dim3(256), 0, st, g); break;             \
    case 64: hipLaunchKernelGGL(K<64>, grid, dim3(256), 0, st, g); break;             \
    default: hipLaunchKernelGGL(K<128>, grid, dim3(256), 0, st, g);                   \
  }

hipError_t launch_lora_shrink_b(const LoraArgs& g, hipStream_t st) {
  const dim3 grid((unsigned)g.splits, (unsigned)g.R.max_units);
  HM_LORA_RANKS(k_lora_shrink_b, grid)
  return hipGetLastError();
}

hipError_t launch_lora_expand_a(const LoraArgs& g, hipStream_t st) {
  const dim3 grid((unsigned)((g.K + kLoraSlab - 1) / kLoraSlab),
                  (unsigned)(g.R.max_units + (g.base != g.y ? (g.M + kLoraUnit - 1) / kLoraUnit : 0)));
  HM_LORA_RANKS(k_lora_expand_a, grid)
  return hipGetLastError();
}

template <bool DB>
static void outer(const LoraArgs& g, hipStream_t st) {
  const unsigned tiles = (unsigned)(((DB ? g.N : g.K) + 127) / 128);
  if (g.rank <= 16) hipLaunchKernelGGL((k_lora_outer<1, DB>), dim3(tiles, 1, g.L), dim3(256), 0, st, g);
  else if (g.rank <= 32) hipLaunchKernelGGL((k_lora_outer<2, DB>), dim3(tiles, 1, g.L), dim3(256), 0, st, g);
  else hipLaunchKernelGGL((k_lora_outer<4, DB>), dim3(tiles, (g.rank + 63) / 64, g.L), dim3(256), 0, st, g);
}

hipError_t launch_lora_outer(const LoraArgs& g, hipStream_t st) {
  outer<false>(g, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  outer<true>(g, st);
  return hipGetLastError();
}

}  // namespace hm
