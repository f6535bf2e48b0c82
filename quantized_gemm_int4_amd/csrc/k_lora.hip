// Low-rank adapters of many requests beside a shared projection, forward:
//   h[m] = s_e A_e x[m]            (contraction over K: "shrink")
//   y[m] = base[m] + B_e h[m]      (contraction over the rank: "expand")
// for every row m of adapter e = ids[m].  Rows are grouped by adapter and cut
// into units of kLoraUnit rows, which share the loads of their adapter's
// matrices.  Both products run on the bf16 MFMA (rows as columns of the
// result); the rank is far too small for either to be bound by it: the shrink
// reads x once, the expand reads base and writes y once, and few-row calls
// read the adapters.
#include "lora.h"

namespace hm {

// Units from the offsets of the grouped rows (one thread per adapter).
__global__ void __launch_bounds__(512)
k_lora_units(const int32_t* __restrict__ offsets, int L, int32_t* __restrict__ hdr, int32_t* __restrict__ units) {
  __shared__ int sum[512];
  const int e = threadIdx.x;
  int beg = 0, c = 0;
  if (e < L) {
    beg = offsets[e];
    c = offsets[e + 1] - beg;
  }
  const int nu = (c + kLoraUnit - 1) / kLoraUnit;
  sum[e] = nu;
  __syncthreads();
  for (int off = 1; off < 512; off <<= 1) {
    const int v = e >= off ? sum[e - off] : 0;
    __syncthreads();
    sum[e] += v;
    __syncthreads();
  }
  const int first = sum[e] - nu;
  for (int i = 0; i < nu; ++i) {
    int32_t* u = units + 4 * (int64_t)(first + i);
    u[0] = e; u[1] = beg + i * kLoraUnit; u[2] = min(c - i * kLoraUnit, kLoraUnit); u[3] = 0;
  }
  if (e == 511) hdr[0] = sum[e];
}

// grid (splits, units): the block's waves split the block's K range; their
// sums meet in LDS and are added in wave order.
template <int RP>
__global__ void __launch_bounds__(256) k_lora_shrink(LoraArgs g) {
  constexpr int RB = RP / 16, LD = RP + 4;
  __shared__ float red[4][kLoraUnit][LD];
  const int u = blockIdx.y;
  if (u >= g.R.hdr[0]) return;
  const int32_t* un = g.R.units + 4 * (int64_t)u;
  const int e = un[0], first = un[1], count = un[2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const int64_t steps = g.K / 32, waves = 4 * (int64_t)g.splits, wi = (int64_t)blockIdx.x * 4 + wave;
  const int64_t s0 = steps * wi / waves, s1 = steps * (wi + 1) / waves;
  const uint16_t* xp[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) xp[t] = g.x + (int64_t)g.R.rows[first + min(16 * t + c, count - 1)] * g.K + 8 * q;
  const uint16_t* ap[RB];        // rows past the rank repeat its last one; their results are not kept
#pragma unroll
  for (int i = 0; i < RB; ++i) ap[i] = g.a + ((int64_t)e * g.rank + min(16 * i + c, g.rank - 1)) * g.K + 8 * q;
  f32x4_t acc[2][RB];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < RB; ++i) acc[t][i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int64_t s = s0; s < s1; ++s) {
    u32x4_t xv[2], av[RB];
#pragma unroll
    for (int t = 0; t < 2; ++t) xv[t] = ld16(xp[t] + 32 * s);
#pragma unroll
    for (int i = 0; i < RB; ++i) av[i] = ld16(ap[i] + 32 * s);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t) acc[t][i] = mfma_bf16(av[i], xv[t], acc[t][i]);
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < RB; ++i) *reinterpret_cast<f32x4_t*>(&red[wave][16 * t + c][16 * i + 4 * q]) = acc[t][i];
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

// grid (column slabs, units + groups of rows without an adapter): y = base +
// B_e h for the unit's rows and the slab's columns.  Lane (c, q) of a wave's
// 64-column group supplies column n0 + 16 (c / 4) + 4 b + c % 4 to MFMA b, so
// that it ends up with the 16 consecutive columns n0 + 16 q + 4 b + v of row c.
template <int RP>
__global__ void __launch_bounds__(256) k_lora_expand(LoraArgs g) {
  using RS = RankSteps<RP>;
  constexpr int half = RP == 16 ? 1 : RP / 32;
  const int64_t c0 = (int64_t)blockIdx.x * kLoraSlab, c1 = min(c0 + kLoraSlab, g.N);
  if (blockIdx.y >= g.R.max_units) {
    copy_rest(g, (blockIdx.y - g.R.max_units) * kLoraUnit, g.N, c0, c1, g.h && blockIdx.x == 0);
    return;
  }
  const int u = blockIdx.y;
  if (u >= g.R.hdr[0]) return;
  const int32_t* un = g.R.units + 4 * (int64_t)u;
  const int e = un[0], first = un[1], count = un[2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  int64_t m[2];
  u32x4_t hf[2][RS::S];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    m[t] = g.R.rows[first + min(16 * t + c, count - 1)];
    load_h_operand<RP>(g.part, g.splits, g.M, g.rank, m[t], q, hf[t]);
  }
  if (g.h && g.part != g.h && blockIdx.x == 0 && wave == 0) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      for (int r0 = 8 * q; r0 < g.rank; r0 += 32) {
        float v[8];
        load_h8(g.part, g.splits, g.M, g.rank, m[t], r0, v);
        if (16 * t + c < count) {
          float4* o = reinterpret_cast<float4*>(g.h + m[t] * g.rank + r0);
          o[0] = make_float4(v[0], v[1], v[2], v[3]);
          o[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
  }
  const uint16_t* B = g.b + (int64_t)e * g.N * g.rank;
  for (int64_t n0 = c0 + 64 * wave; n0 < c1; n0 += 256) {
    f32x4_t acc[2][4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int64_t n = min(n0 + 16 * (c >> 2) + 4 * b + (c & 3), g.N - 1);
#pragma unroll
      for (int t = 0; t < 2; ++t) acc[t][b] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < half; ++s) {
        const int r0 = RS::r0(s, q);
        u32x4_t bv = {0u, 0u, 0u, 0u};
        if (r0 < g.rank) bv = ld16(B + n * g.rank + r0);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          acc[t][b] = mfma_bf16(bv, hf[t][s], acc[t][b]);
          if (RP != 16) acc[t][b] = mfma_bf16(bv, hf[t][half + s], acc[t][b]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (16 * t + c >= count) continue;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int64_t n = n0 + 16 * q + 8 * p;
        if (n >= g.N) continue;
        const float v[8] = {acc[t][2 * p][0], acc[t][2 * p][1], acc[t][2 * p][2], acc[t][2 * p][3],
                            acc[t][2 * p + 1][0], acc[t][2 * p + 1][1], acc[t][2 * p + 1][2], acc[t][2 * p + 1][3]};
        add_store8(g.base ? g.base + m[t] * g.N : nullptr, g.y + m[t] * g.N, n, g.N, v);
      }
    }
  }
}

hipError_t launch_lora_units(const int32_t* offsets, int L, int32_t* hdr, int32_t* units, hipStream_t st) {
  hipLaunchKernelGGL(k_lora_units, dim3(1), dim3(512), 0, st, offsets, L, hdr, units);
  return hipGetLastError();
}

hipError_t launch_lora_shrink(const LoraArgs& g, hipStream_t st) {
  const dim3 grid((unsigned)g.splits, (unsigned)g.R.max_units);
  switch (lora_rp(g.rank)) {
    case 16: hipLaunchKernelGGL(k_lora_shrink<16>, grid, dim3(256), 0, st, g); break;
    case 32: hipLaunchKernelGGL(k_lora_shrink<32>, grid, dim3(256), 0, st, g); break;
    case 64: hipLaunchKernelGGL(k_lora_shrink<64>, grid, dim3(256), 0, st, g); break;
    default: hipLaunchKernelGGL(k_lora_shrink<128>, grid, dim3(256), 0, st, g);
  }
  return hipGetLastError();
}

hipError_t launch_lora_expand(const LoraArgs& g, hipStream_t st) {
  const bool rest = g.base != g.y || g.h;
  const dim3 grid((unsigned)((g.N + kLoraSlab - 1) / kLoraSlab),
                  (unsigned)(g.R.max_units + (rest ? (g.M + kLoraUnit - 1) / kLoraUnit : 0)));
  switch (lora_rp(g.rank)) {
    case 16: hipLaunchKernelGGL(k_lora_expand<16>, grid, dim3(256), 0, st, g); break;
    case 32: hipLaunchKernelGGL(k_lora_expand<32>, grid, dim3(256), 0, st, g); break;
    case 64: hipLaunchKernelGGL(k_lora_expand<64>, grid, dim3(256), 0, st, g); break;
    default: hipLaunchKernelGGL(k_lora_expand<128>, grid, dim3(256), 0, st, g);
  }
  return hipGetLastError();
}

}  // namespace hm
