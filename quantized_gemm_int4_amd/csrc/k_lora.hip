// Low-rank adapters of many requests beside a shared projection.  For every
// row m of adapter e = ids[m]:
//   forward    h[m] = s_e A_e x[m]           y[m] = base[m] + B_e h[m]
//   gradient   g[m] = s_e B_e^T dy[m]        dx[m] = dx_base[m] + A_e^T g[m]
// that is, one contraction of long rows to the rank ("shrink") and one
// product back ("expand"), the gradient's with the transposed matrices
// (TRANS).  Rows are grouped by adapter into units that share the loads of
// their adapter's matrices.  Both products run on the bf16 MFMA with the rows
// as columns of the result; the rank is far too small for either to be bound
// by it: the shrink reads its rows once, the expand reads base and writes y
// once, and calls of few rows read the adapters.  An MFMA operand wants eight
// consecutive values of the contracted axis per lane; where that axis is the
// strided one in memory (TRANS) a lane loads eight rows of a few neighbouring
// columns and transposes them in its registers, each column being one MFMA's.
#include "lora.h"
#include "sort.h"

namespace hm {

// Grouping of the rows by adapter in one launch: every block counts all ids
// (and those before its chunk of C rows), so that each can place its own
// chunk without a pass in between; block 0 writes the units.  Counting is
// cheap next to the call (4 bytes a row and block, at most kLoraPlanBlocks
// blocks, against rows of thousands of bytes) and a second launch is not.
__global__ void __launch_bounds__(kSortThreads)
k_lora_plan(const int32_t* __restrict__ ids, int64_t M, int L, int64_t C, int U, int64_t max_units,
            int32_t* __restrict__ units, int32_t* __restrict__ rows, int32_t* __restrict__ firsts) {
  __shared__ int hist[kSortWaves][512];
  __shared__ int before[512], after[512], base[512], uend[512];
  __shared__ int wsum[8];
  const int tid = threadIdx.x, lane = tid & 63;
  for (int i = tid; i < 512; i += kSortThreads) before[i] = after[i] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * C, hi = min(lo + C, M);
  for (int64_t p0 = 0; p0 < M; p0 += kSortThreads) {          // C is a multiple of kSortThreads
    int* cnt = p0 < lo ? before : after;
    const int e = p0 + tid < M ? ids[p0 + tid] : -1;
    const bool ok = e >= 0 && e < L;
    const uint64_t m = __ballot(ok);
    if (!m) continue;
    // rows of a prompt carry one id: one addition for the wave
    const int first = __shfl(e, __builtin_ctzll(m), 64);
    if (__ballot(ok && e == first) == m) {
      if (lane == 0) atomicAdd(&cnt[first], __popcll(m));
    } else if (ok) {
      atomicAdd(&cnt[e], 1);
    }
  }
  __syncthreads();
  const int total = tid < 512 ? before[tid] + after[tid] : 0;
  const int nu = (total + U - 1) / U;
  const int ue = block_scan512(nu, wsum);
  if (tid < 512) {
    uend[tid] = ue;
    base[tid] = (ue - nu) * U + before[tid];                  // rows land in their units' slots
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    if (tid <= L) firsts[tid] = tid ? uend[tid - 1] : 0;
    for (int u = tid; u < max_units; u += kSortThreads) {
      int e = 0;                                              // first adapter whose units end after u
      for (int step = 256; step >= 1; step >>= 1)
        if (e + step <= 511 && uend[e + step - 1] <= u) e += step;
      const int i = u - (e ? uend[e - 1] : 0);
      const bool used = u < uend[511];
      units[2 * u] = used ? e : 0;
      units[2 * u + 1] = used ? min(before[e] + after[e] - i * U, U) : 0;
    }
  }
  sort_range<false>(ids, lo, hi, L, base, hist, rows, nullptr);
}

// Rows first .. first + U - 1 of unit u: its adapter, and those rows in LDS.
// Direct calls (few rows, no grouping launch): the block of row u takes row u
// and the next 15 rows of the same adapter if 16, 32, ... rows of it come
// before; other blocks get count 0.  Returns the count; -1 (direct) for a row
// without an adapter.  Must be reached by every thread of the block.
template <int U, bool DIRECT>
__device__ __forceinline__ int find_unit(const LoraArgs& g, int u, int first, int* e, int* rows) {
  if constexpr (DIRECT) {
    const int lane = threadIdx.x & 63;
    const int id = lane < g.M ? g.ids[lane] : -1;             // M <= 64: one wave's ballot has them all
    *e = __builtin_amdgcn_readlane(id, u);
    if (*e < 0 || *e >= g.L) return -1;
    const uint64_t m = __ballot(id == *e);
    const int before = __popcll(m & ((1ull << u) - 1));
    if (before % 16) return 0;
    const int rank = __popcll(m & (lane ? (~0ull >> (64 - lane)) : 0ull)) - before;
    if (threadIdx.x < 64 && id == *e && rank >= 0 && rank < 16) rows[rank] = lane;
    __syncthreads();
    return min(__popcll(m) - before, 16);
  } else {
    *e = g.R.units[2 * u];
    const int count = min(g.R.units[2 * u + 1] - first, U);
    if ((int)threadIdx.x < count) rows[threadIdx.x] = g.R.rows[(int64_t)u * g.R.unit_rows + first + threadIdx.x];
    __syncthreads();
    return count;
  }
}

// Waves of a contracting block.
constexpr int shrink_waves(int t) { return t == 1 ? 4 : 8; }

// grid (splits, units x blocks of 16 T rows): the block's waves split the
// block's range of the contracted axis; their sums meet in LDS and are added
// in wave order.  A wave loads NB steps of 32 values before the first MFMA.
template <int RP, int T, bool DIRECT, bool TRANS>
__global__ void __launch_bounds__(64 * shrink_waves(T)) k_lora_shrink(LoraArgs g) {
  constexpr int RB = RP / 16, LD = RP + 4, U = 16 * T, NW = shrink_waves(T);
  constexpr int NB = TRANS ? (RP >= 64 ? 2 : 4) : (T + RB > 8 ? 2 : (T + RB > 4 ? 4 : 8));
  // LDS images of the sums: one per wave while that is small, else one for several waves in turn
  constexpr int FIT = 70 * 1024 / (U * LD * 4);
  constexpr int BUF = FIT >= NW ? NW : (FIT >= NW / 2 ? NW / 2 : (FIT >= NW / 4 ? NW / 4 : 1));
  __shared__ float red[BUF][U][LD];
  __shared__ int rows[U];
  const int sub = DIRECT ? 1 : g.R.unit_rows / U;
  int e;
  const int count = find_unit<U, DIRECT>(g, blockIdx.y / sub, blockIdx.y % sub * U, &e, rows);
  if (count <= 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const int64_t len = TRANS ? g.N : g.K;
  const int steps = (int)(len / 32), waves = NW * g.splits, wi = (int)blockIdx.x * NW + wave;
  const int s0 = (int)((int64_t)steps * wi / waves), s1 = (int)((int64_t)steps * (wi + 1) / waves);
  const uint16_t* zp[T];
#pragma unroll
  for (int t = 0; t < T; ++t) zp[t] = g.z + (int64_t)rows[min(16 * t + c, count - 1)] * len + 8 * q;
  // A: lane c supplies rank row 16 i + c to MFMA i (rows past the rank repeat its last one; their results are not
  // kept).  B, transposed: rank column RB c + i.
  const uint16_t* ap[TRANS ? 1 : RB];
  if constexpr (TRANS) {
    ap[0] = g.b + ((int64_t)e * g.N + 8 * q) * g.rank + RB * c;
  } else {
#pragma unroll
    for (int i = 0; i < RB; ++i) ap[i] = g.a + ((int64_t)e * g.rank + min(16 * i + c, g.rank - 1)) * g.K + 8 * q;
  }
  const int in_rank = RB * c < g.rank ? 8 : 0;
  f32x4_t acc[T][RB];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int i = 0; i < RB; ++i) acc[t][i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  auto batch = [&](int s, auto steps_c) __attribute__((always_inline)) {
    constexpr int n = decltype(steps_c)::value;
    u32x4_t zv[n][T], av[n][TRANS ? 1 : RB];
    Cols8<TRANS ? RB : 1> bv[n];
#pragma unroll
    for (int j = 0; j < n; ++j) {
#pragma unroll
      for (int t = 0; t < T; ++t) zv[j][t] = TRANS ? ld8(zp[t] + 32 * (s + j)) : ld16(zp[t] + 32 * (s + j));
      if constexpr (TRANS) {
        bv[j].load(ap[0] + (int64_t)32 * (s + j) * g.rank, g.rank, in_rank);
      } else {
#pragma unroll
        for (int i = 0; i < RB; ++i) av[j][i] = ld16(ap[i] + 32 * (s + j));
      }
    }
    loads_first();
#pragma unroll
    for (int j = 0; j < n; ++j)
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const u32x4_t a = TRANS ? bv[j].operand(i) : av[j][TRANS ? 0 : i];
#pragma unroll
        for (int t = 0; t < T; ++t) acc[t][i] = mfma_bf16(a, zv[j][t], acc[t][i]);
      }
  };
  int s = s0;
  for (; s + NB <= s1; s += NB) batch(s, Int<NB>{});
  if constexpr (NB > 4)
    if (s + 4 <= s1) { batch(s, Int<4>{}); s += 4; }
  if constexpr (NB > 2)
    if (s + 2 <= s1) { batch(s, Int<2>{}); s += 2; }
  if (s < s1) batch(s, Int<1>{});
  if (TRANS && wi == waves - 1 && len % 32) {                 // the columns behind the last whole step
    const int64_t n = 32 * (int64_t)steps + 8 * q, left = len - n;
    Cols8<TRANS ? RB : 1> bv;
    bv.load(ap[0] + (int64_t)32 * steps * g.rank, g.rank, min(in_rank, (int)max(left, (int64_t)0)));
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const u32x4_t zv = left > 0 ? ld8_tail(zp[t] - 8 * q, n, len) : (u32x4_t){0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < RB; ++i) acc[t][i] = mfma_bf16(bv.operand(i), zv, acc[t][i]);
    }
  }
#pragma unroll
  for (int w = 0; w < NW / BUF; ++w) {
    if (wave / BUF == w) {
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            float* p = &red[wave % BUF][16 * t + c][TRANS ? RB * (4 * q + v) + i : 16 * i + 4 * q + v];
            *p = w == 0 ? acc[t][i][v] : *p + acc[t][i][v];
          }
    }
    __syncthreads();
  }
  const float sc = g.scales[e];
  float* out = g.part + (int64_t)blockIdx.x * g.M * g.rank;
  for (int i = threadIdx.x; i < count * (RP / 4); i += 64 * NW) {
    const int row = i / (RP / 4), r = 4 * (i % (RP / 4));
    if (r >= g.rank) continue;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(&red[0][row][r]);
#pragma unroll
    for (int w = 1; w < BUF; ++w) v += *reinterpret_cast<const f32x4_t*>(&red[w][row][r]);
    *reinterpret_cast<f32x4_t*>(out + (int64_t)rows[row] * g.rank + r) = v * sc;
  }
}

// Row m without an adapter, columns [c0, c1) of n: y = base (zeros without
// one); one wave.
__device__ __forceinline__ void copy_row(const LoraArgs& g, int64_t m, int64_t n, int64_t c0, int64_t c1, bool zero_h) {
  const int lane = threadIdx.x & 63;
  if (g.base != g.y)
    for (int64_t c = c0 + 8 * lane; c < c1; c += 512)
      st8_tail(g.y + m * n, c, n, g.base ? ld8_tail(g.base + m * n, c, n) : (u32x4_t){0u, 0u, 0u, 0u});
  if (zero_h)
    for (int r = lane; r < g.rank; r += 64) g.h[m * g.rank + r] = 0.f;
}

// One block per (256 columns, group of units, or 64 rows of which those
// without an adapter are copied): y = base + B_e h.  A wave holds 64 columns
// of B_e in registers while its group's units have the same adapter and takes
// their rows 16 at a time.  Lane c supplies column 32 (b / 2) + 8 (c / 4) + 4
// (b % 2) + c % 4 to MFMA b (TRANS: column 32 (c % 4 / 2) + 8 (c / 4) + 4 (c %
// 2) + b) and so ends up, in quarter q, with columns 8 q .. + 7 and 32 + 8 q
// .. + 7 of row c: four lanes write 64 consecutive bytes.  Blocks go round
// the XCDs one by one, so block id i takes columns i % 8 + 8 k: each XCD sees
// an eighth of B_e, which stays in its L2 from group to group.
template <int RP, int T, bool DIRECT, bool TRANS>
__global__ void __launch_bounds__(256) k_lora_expand(LoraArgs g) {
  constexpr int S = RP == 16 ? 1 : RP / 16, HALF = RP == 16 ? 1 : RP / 32, U = 16 * T, LDH = 2 * RP + 8;
  __shared__ __align__(16) uint16_t hs[2][U][LDH];            // a row's h: RP values hi, RP values lo
  __shared__ int rows[2][U];
  const int64_t N = TRANS ? g.K : g.N;
  const int per = (int)((N + 8 * kLoraCols - 1) / (8 * kLoraCols));       // column slabs per XCD
  const uint32_t id = blockIdx.x >> 3;
  const int gi = (int)(id / per), slab = (int)(blockIdx.x & 7) + 8 * (int)(id % per);
  const int64_t c0 = (int64_t)slab * kLoraCols, c1 = min(c0 + kLoraCols, N);
  if (c0 >= N) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const bool keep = !TRANS && g.h && slab == 0;
  const int groups = DIRECT ? (int)g.M : (int)((g.R.max_units + g.group - 1) / g.group);
  if (!DIRECT && gi >= groups) {
    const int64_t m0 = (int64_t)(gi - groups) * 64;
    for (int64_t m = m0 + wave; m < min(m0 + 64, g.M); m += 4) {
      const int e = g.ids[m];
      if (e < 0 || e >= g.L) copy_row(g, m, N, c0, c1, keep);
    }
    return;
  }
  const int64_t n0 = c0 + 64 * wave;
  // rank column of MFMA step s (of 32 over [hi | lo]) that quarter q supplies first; RP = 16: one step, 0-1 hi, 2-3 lo
  auto rank0 = [q](int s) { return RP == 16 ? 8 * (q & 1) : 32 * s + 8 * q; };
  u32x4_t bv[TRANS ? 1 : 4][HALF], yv[T][2];
  Cols8<4> cv[TRANS ? HALF : 1];
  int have = -1;
  const int u0 = DIRECT ? gi : gi * g.group, un = DIRECT ? gi + 1 : (int)min((int64_t)u0 + g.group, g.R.max_units);
  for (int u = u0; u < un; ++u) {
    int e, *rw = rows[u & 1];
    uint16_t(*hu)[LDH] = hs[u & 1];
    const int count = find_unit<U, DIRECT>(g, u, 0, &e, rw);
    if (count <= 0) {
      if (DIRECT && count < 0 && wave == 0) copy_row(g, u, N, c0, c1, keep);
      return;                                                 // units behind the last used one are empty too
    }
    if (n0 < N) {
      if (e != have) {
        have = e;
        if constexpr (TRANS) {
          const uint16_t* A = g.a + (int64_t)e * g.rank * g.K + n0 + 32 * ((c >> 1) & 1) + 8 * (c >> 2) + 4 * (c & 1);
#pragma unroll
          for (int s = 0; s < HALF; ++s) cv[s].load(A + (int64_t)rank0(s) * g.K, g.K, rank0(s) < g.rank ? 8 : 0);
        } else {
          const uint16_t* B = g.b + (int64_t)e * g.N * g.rank;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int64_t n = min(n0 + 32 * (b >> 1) + 8 * (c >> 2) + 4 * (b & 1) + (c & 3), N - 1);
#pragma unroll
            for (int s = 0; s < HALF; ++s) {
              bv[b][s] = (u32x4_t){0u, 0u, 0u, 0u};
              if (rank0(s) < g.rank) bv[b][s] = ld16(B + n * g.rank + rank0(s));
            }
          }
        }
      }
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const uint16_t* br = g.base + (int64_t)rw[min(16 * t + c, count - 1)] * N;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int64_t n = n0 + 32 * p + 8 * q;
          yv[t][p] = (u32x4_t){0u, 0u, 0u, 0u};
          if (g.base && n < N) yv[t][p] = ld8_tail(br, n, N);
        }
      }
    }
    loads_first();
    // h of the unit's rows: the splits' sums in split order, as two bf16 terms
    auto stage = [&](auto max_splits) __attribute__((always_inline)) {
      constexpr int MS = decltype(max_splits)::value;
      for (int i = threadIdx.x; i < count * (RP / 4); i += 256) {
        const int row = i / (RP / 4), r0 = 4 * (i % (RP / 4));
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
        if (r0 < g.rank) {
          const int64_t at = (int64_t)rw[row] * g.rank + r0;
          f32x4_t p[MS];
#pragma unroll
          for (int s = 0; s < MS; ++s)
            p[s] = *reinterpret_cast<const f32x4_t*>(g.part + (int64_t)min(s, g.splits - 1) * g.M * g.rank + at);
          loads_first();
#pragma unroll
          for (int s = 0; s < MS; ++s)
            if (s < g.splits) v += p[s];
          if (keep && g.part != g.h) *reinterpret_cast<f32x4_t*>(g.h + at) = v;
        }
        u32x2_t hi, lo;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t h2, l2;
          split2(v[2 * k], v[2 * k + 1], &h2, &l2);
          hi[k] = h2;
          lo[k] = l2;
        }
        *reinterpret_cast<u32x2_t*>(&hu[row][r0]) = hi;
        *reinterpret_cast<u32x2_t*>(&hu[row][RP + r0]) = lo;
      }
    };
    if (g.splits == 1) stage(Int<1>{});
    else if (T > 1 || g.splits <= 4) stage(Int<4>{});
    else stage(Int<kLoraMaxSplits>{});
    __syncthreads();
    if (n0 >= N) continue;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if (16 * t >= count) break;
      const uint16_t* hr = hu[min(16 * t + c, count - 1)] + 8 * q;
      u32x4_t hf[S];
#pragma unroll
      for (int s = 0; s < S; ++s) hf[s] = ld16(hr + 32 * s);
      f32x4_t acc[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        acc[b] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const u32x4_t a = TRANS ? cv[TRANS ? s % HALF : 0].operand(b) : bv[TRANS ? 0 : b][s % HALF];
          acc[b] = mfma_bf16(a, hf[s], acc[b]);
        }
      }
      if (16 * t + c < count) {
        uint16_t* yr = g.y + (int64_t)rw[16 * t + c] * N;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int64_t n = n0 + 32 * p + 8 * q;
          u32x4_t o;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float lo = TRANS ? acc[2 * (k & 1)][2 * p + (k >> 1)] : acc[2 * p + (k >> 1)][2 * (k & 1)];
            const float hi = TRANS ? acc[2 * (k & 1) + 1][2 * p + (k >> 1)] : acc[2 * p + (k >> 1)][2 * (k & 1) + 1];
            o[k] = pack_bf16(lo_bf16(yv[t][p][k]) + lo, hi_bf16(yv[t][p][k]) + hi);
          }
          if (n < N) st8_tail(yr, n, N, o);
        }
      }
    }
  }
}

hipError_t launch_lora_plan(const int32_t* ids, int64_t M, int L, int unit_rows, int64_t max_units, int32_t* units,
                            int32_t* rows, int32_t* first, hipStream_t st) {
  const int64_t per = (M + kLoraPlanBlocks - 1) / kLoraPlanBlocks;
  const int64_t C = (per + kSortThreads - 1) / kSortThreads * kSortThreads;
  hipLaunchKernelGGL(k_lora_plan, dim3((unsigned)((M + C - 1) / C)), dim3(kSortThreads), 0, st, ids, M, L, C,
                     unit_rows, max_units, units, rows, first);
  return hipGetLastError();
}

template <int RP, bool TRANS>
static void run_shrink(const LoraArgs& g, bool direct, hipStream_t st) {
  const int t = direct || g.R.unit_rows == 16 ? 1 : 2;
  const dim3 grid((unsigned)g.splits, (unsigned)(direct ? g.M : g.R.max_units * (g.R.unit_rows / (16 * t))));
  const dim3 block(64u * (unsigned)shrink_waves(t));
  if constexpr (!TRANS) {
    if (direct) hipLaunchKernelGGL((k_lora_shrink<RP, 1, true, false>), grid, block, 0, st, g);
    else if (t == 1) hipLaunchKernelGGL((k_lora_shrink<RP, 1, false, false>), grid, block, 0, st, g);
  }
  if (t == 2) hipLaunchKernelGGL((k_lora_shrink<RP, 2, false, TRANS>), grid, block, 0, st, g);
}

template <int RP, bool TRANS>
static void run_expand(const LoraArgs& g, bool direct, hipStream_t st) {
  const int64_t cols = TRANS ? g.K : g.N;
  const int64_t per = (cols + 8 * kLoraCols - 1) / (8 * kLoraCols);
  const bool rest = g.base != g.y || (!TRANS && g.h);
  const int64_t groups = direct ? g.M : (g.R.max_units + g.group - 1) / g.group + (rest ? (g.M + 63) / 64 : 0);
  const dim3 grid((unsigned)(8 * per * groups));
  if constexpr (!TRANS) {
    if (direct) hipLaunchKernelGGL((k_lora_expand<RP, 1, true, false>), grid, dim3(256), 0, st, g);
    else if (g.R.unit_rows == 16) hipLaunchKernelGGL((k_lora_expand<RP, 1, false, false>), grid, dim3(256), 0, st, g);
    else if (g.R.unit_rows == 32) hipLaunchKernelGGL((k_lora_expand<RP, 2, false, false>), grid, dim3(256), 0, st, g);
  }
  if (!direct && g.R.unit_rows == 64) hipLaunchKernelGGL((k_lora_expand<RP, 4, false, TRANS>), grid, dim3(256), 0, st, g);
}

#define HM_LORA_RANKS(F)                                                          \
  switch (lora_rp(g.rank)) {                                                      \
    case 16: trans ? F<16, true>(g, direct, st) : F<16, false>(g, direct, st); break; \
    case 32: trans ? F<32, true>(g, direct, st) : F<32, false>(g, direct, st); break; \
    case 64: trans ? F<64, true>(g, direct, st) : F<64, false>(g, direct, st); break; \
    default: trans ? F<128, true>(g, direct, st) : F<128, false>(g, direct, st);  \
  }

hipError_t launch_lora_shrink(const LoraArgs& g, bool direct, bool trans, hipStream_t st) {
  HM_LORA_RANKS(run_shrink)
  return hipGetLastError();
}

hipError_t launch_lora_expand(const LoraArgs& g, bool direct, bool trans, hipStream_t st) {
  HM_LORA_RANKS(run_expand)
  return hipGetLastError();
}

}  // namespace hm
