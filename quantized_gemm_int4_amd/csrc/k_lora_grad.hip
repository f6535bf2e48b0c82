// Gradient of the low-rank adapters to their matrices: for every adapter e
// the sums over its rows m
//   da_e = sum_m g[m] x[m]^T,   db_e = sum_m dy[m] h[m]^T
// (g and dx are k_lora.hip's).  The contraction runs over the rows, which are
// the strided axis of x and dy: a lane loads eight rows of eight neighbouring
// columns and transposes them in its registers, each column being one MFMA's
// operand.  g and h are small; a packing pass (k_lora_dx's) brings them into operand order
// once (as three bf16 terms), because every column tile reads them again (read
// in their own order, 64 cache lines an access, they bound the kernel: m =
// 8192, n = 14336, k = 4096, rank 32 189 us; now 73 us, 4.1 TB/s of dy and x).
#include "lora.h"

namespace hm {

__device__ __forceinline__ int chunk_units(const LoraGradArgs& g) {
  return (g.R.first[g.L] + g.chunks - 1) / g.chunks;
}

// One block per (128-column tile of dy or x, chunk of units, rank chunk of 16
// RB): one adapter of the chunk after the other.  Block id i takes tile i % 8
// + 8 k, its rank chunks side by side: they read the same rows at about the
// same time through one XCD's L2.  The waves take its 32-row
// steps in turn; their sums meet in LDS, in wave order.  An adapter that
// reaches beyond the chunk leaves a partial sum: slot 2 j if it began before
// chunk j, else 2 j + 1.
template <int RP, int RB, bool db>
__device__ __forceinline__ void outer_tile(const LoraGradArgs& g, int64_t k0, int chunk, int r00, float (*red)[132]) {
  constexpr int RC = 16 * RB;
  const int64_t n = db ? g.N : g.K;
  const uint16_t* z = db ? g.dy : g.x;
  const uint16_t* f = (db ? g.ht : g.gt) + r00 * 32 + 8 * (threadIdx.x & 63);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const int per = chunk_units(g), lo_u = chunk * per, hi_u = min(lo_u + per, g.R.first[g.L]);
  const int64_t col = k0 + 8 * c;
  for (int ua = lo_u; ua < hi_u;) {
    const int e = g.R.units[2 * ua], e0 = g.R.first[e], e1 = g.R.first[e + 1], ub = min(e1, hi_u);
    f32x4_t acc[8][RB];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < RB; ++i) acc[j][i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    // Two steps ahead the row numbers are on their way, one step ahead the rows: a gathered load waits for two trips
    // to memory otherwise (m = 8192: 113 us).
    struct Rows { int r[8], count; };
    auto fetch_rows = [&](int s) __attribute__((always_inline)) {
      Rows R;
      const int32_t* p = g.R.rows + 32 * (int64_t)s;          // a unit's slots: two steps of 32
      const int4 lo = *reinterpret_cast<const int4*>(p + 8 * q), hi = *reinterpret_cast<const int4*>(p + 8 * q + 4);
      R.r[0] = lo.x; R.r[1] = lo.y; R.r[2] = lo.z; R.r[3] = lo.w;
      R.r[4] = hi.x; R.r[5] = hi.y; R.r[6] = hi.z; R.r[7] = hi.w;
      R.count = g.R.units[2 * (s >> 1) + 1] - 32 * (s & 1);
      return R;
    };
    Cols8<8> next;
    auto fetch_z = [&](const Rows& R) __attribute__((always_inline)) {
      const int first = __builtin_amdgcn_readfirstlane(R.r[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // rows behind the unit's last read the step's first and count as 0, as their g and h are
        const bool in = 8 * q + i < R.count;
        const int64_t m = in ? R.r[i] : first;
        u32x4_t v = {0u, 0u, 0u, 0u};
        if (R.count > 0 && col < n) v = ld8_tail(z + m * n, col, n);
#pragma unroll
        for (int k = 0; k < 4; ++k) next.w[i][k] = in ? v[k] : 0u;
      }
    };
    const int s_end = 2 * ub;
    int s = 2 * ua + wave;
    Rows R{};
    if (s < s_end) {
      R = fetch_rows(s);
      fetch_z(R);
      if (s + 4 < s_end) R = fetch_rows(s + 4);
    }
    for (; s < s_end; s += 4) {
      const Cols8<8> zv = next;
      u32x4_t fv[kTerms][RB];
      const uint16_t* fu = f + (int64_t)s * kTerms * RP * 32;
#pragma unroll
      for (int i = 0; i < kTerms; ++i)
#pragma unroll
        for (int k = 0; k < RB; ++k) fv[i][k] = ld16(fu + RP * 32 * i + 512 * k);
      const int count = g.R.units[2 * (s >> 1) + 1] - 32 * (s & 1);
      if (s + 4 < s_end) {
        fetch_z(R);
        if (s + 8 < s_end) R = fetch_rows(s + 8);
      }
      loads_first();
      if (count <= 0) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const u32x4_t zo = zv.operand(j);
#pragma unroll
        for (int k = 0; k < RB; ++k)
#pragma unroll
          for (int i = 0; i < kTerms; ++i)
            acc[j][k] = db ? mfma_bf16(fv[i][k], zo, acc[j][k]) : mfma_bf16(zo, fv[i][k], acc[j][k]);
      }
    }
    // db: the lane holds column 8 c + j, rank 16 k + 4 q + v; da: rank 16 k + c, column 8 (4 q + v) + j
    for (int w = 0; w < 4; ++w) {
      if (w == wave)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int k = 0; k < RB; ++k)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              float* p = db ? &red[16 * k + 4 * q + v][8 * c + j] : &red[16 * k + c][8 * (4 * q + v) + j];
              *p = w == 0 ? acc[j][k][v] : *p + acc[j][k][v];
            }
      __syncthreads();
    }
    const bool whole = e0 >= lo_u && e1 <= hi_u;
    float* part = g.sums + (int64_t)(2 * chunk + (e0 < lo_u ? 0 : 1)) * g.rank * (g.K + g.N);
    for (int i = threadIdx.x; i < 128 * RC / 8; i += 256) {
      int64_t at;
      float o[8];
      if (db) {
        const int cc = i / (RC / 8), r = 8 * (i % (RC / 8));
        if (k0 + cc >= n || r00 + r >= g.rank) continue;
        at = (k0 + cc) * g.rank + r00 + r;
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = red[r + k][cc];
      } else {
        const int r = i / 16, cc = 8 * (i % 16);
        if (r00 + r >= g.rank) continue;
        at = (int64_t)(r00 + r) * n + k0 + cc;
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = red[r][cc + k];
      }
      if (whole) {
        st16((db ? g.db : g.da) + (int64_t)e * n * g.rank + at,
             (u32x4_t){pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7])});
      } else {
        float* p = part + (db ? (int64_t)g.rank * g.K : 0) + at;
        *reinterpret_cast<f32x4_t*>(p) = (f32x4_t){o[0], o[1], o[2], o[3]};
        *reinterpret_cast<f32x4_t*>(p + 4) = (f32x4_t){o[4], o[5], o[6], o[7]};
      }
    }
    __syncthreads();
    ua = ub;
  }
}

template <int RP, int RB>
__global__ void __launch_bounds__(256, 2) k_lora_outer(LoraGradArgs g) {
  constexpr int RCS = RP / (16 * RB);
  __shared__ float red[16 * RB][132];
  const int tiles_n = (int)((g.N + 127) / 128), tiles = tiles_n + (int)(g.K / 128), per = (tiles + 7) / 8;
  const int id = blockIdx.x >> 3, r00 = id % RCS * 16 * RB, at = id / RCS;
  const int tile = at % per * 8 + (int)(blockIdx.x & 7), chunk = at / per;
  if (tile < tiles_n) outer_tile<RP, RB, true>(g, 128 * (int64_t)tile, chunk, r00, red);
  else if (tile < tiles) outer_tile<RP, RB, false>(g, 128 * (int64_t)(tile - tiles_n), chunk, r00, red);
}

// grid (eight values per thread of an adapter's da and db, adapters): sums of
// the partial sums in chunk order for adapters that reach over chunks.
__global__ void __launch_bounds__(256) k_lora_sums(LoraGradArgs g) {
  const int e = blockIdx.y;
  const int64_t i = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x), na = (int64_t)g.rank * g.K, nb = (int64_t)g.rank * g.N;
  if (i >= na + nb) return;
  const int u0 = g.R.first[e], u1 = g.R.first[e + 1];
  if (u0 == u1) return;                                       // zeros, written beside dx
  const int per = chunk_units(g), j0 = u0 / per, j1 = (u1 - 1) / per;
  if (j0 == j1) return;                                       // written whole
  f32x4_t a = {0.f, 0.f, 0.f, 0.f}, b = {0.f, 0.f, 0.f, 0.f};
  for (int j = j0; j <= j1; ++j) {
    const float* p = g.sums + (int64_t)(2 * j + (j == j0 ? 1 : 0)) * (na + nb) + i;
    a += *reinterpret_cast<const f32x4_t*>(p);
    b += *reinterpret_cast<const f32x4_t*>(p + 4);
  }
  st16(i < na ? g.da + e * na + i : g.db + e * nb + i - na,
       (u32x4_t){pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3])});
}

hipError_t launch_lora_outer(const LoraGradArgs& g, hipStream_t st) {
  const int64_t per = ((g.N + 127) / 128 + g.K / 128 + 7) / 8;
  const int rp = lora_rp(g.rank);
  const dim3 grid((unsigned)(8 * per * g.chunks * (rp == 16 ? 1 : rp / 32)));
  switch (rp) {
    case 16: hipLaunchKernelGGL((k_lora_outer<16, 1>), grid, dim3(256), 0, st, g); break;
    case 32: hipLaunchKernelGGL((k_lora_outer<32, 2>), grid, dim3(256), 0, st, g); break;
    case 64: hipLaunchKernelGGL((k_lora_outer<64, 2>), grid, dim3(256), 0, st, g); break;
    default: hipLaunchKernelGGL((k_lora_outer<128, 2>), grid, dim3(256), 0, st, g);
  }
  return hipGetLastError();
}

hipError_t launch_lora_sums(const LoraGradArgs& g, hipStream_t st) {
  const int64_t per = g.rank * (g.K + g.N) / 8;
  hipLaunchKernelGGL(k_lora_sums, dim3((unsigned)((per + 255) / 256), (unsigned)g.L), dim3(256), 0, st, g);
  return hipGetLastError();
}

}  // namespace hm
