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
  for (int64_t p0 = 0; p0 < M; p0 += 8 * kSortThreads) {
    int id[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t p = p0 + i * kSortThreads + tid;
      id[i] = p < M ? ids[p] : -1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int* cnt = p0 + i * kSortThreads < lo ? before : after; // C is a multiple of kSortThreads
      const int e = id[i];
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
constexpr int shrink_waves(int rp, int t) { return t == 1 || rp == 128 ? 4 : 8; }

// A wave's private LDS image of 64 values of 16 rows: row r's 16-byte chunk k
// (0 .. 7) sits at place k ^ (r & 7) of its 128 bytes, so that both the
// writes (eight lanes per row) and the reads (sixteen rows' chunk) spread over
// the banks.
__device__ __forceinline__ int chunk_at(int r, int k) { return r * 128 + ((k ^ (r & 7)) << 4); }

// grid (splits, units x blocks of 16 T rows): the block's waves split the
// block's range of the contracted axis into steps of 64; their sums meet in
// LDS and are added in wave order.  A load instruction is cheapest when
// neighbouring lanes read neighbouring bytes, while an MFMA operand has a row
// per lane: loaded in operand order, sixteen lanes touch sixteen cache lines
// of 16 bytes each and the address unit, not HBM, sets the pace (m = 8192, k =
// 4096, rank 64: 50 us).  So a wave loads eight whole lines per instruction
// into registers, one step ahead, and passes them through its own LDS image;
// no block barrier.
template <int RP, int T, bool DIRECT, bool TRANS>
__global__ void __launch_bounds__(64 * shrink_waves(RP, T)) k_lora_shrink(LoraArgs g) {
  constexpr int RB = RP / 16, LD = RP + 4, U = 16 * T, NW = shrink_waves(RP, T);
  constexpr int TILES = TRANS ? T : T + RB;                   // 16-row tiles staged per step
  // LDS: the waves' images, then the sums (one per wave while that is small, else one for several waves in turn)
  constexpr int IMG = TILES * 2048, FIT = 72 * 1024 / (U * LD * 4);
  constexpr int BUF = FIT >= NW ? NW : (FIT >= NW / 2 ? NW / 2 : (FIT >= NW / 4 ? NW / 4 : 1));
  constexpr int BYTES = NW * IMG > BUF * U * LD * 4 ? NW * IMG : BUF * U * LD * 4;
  __shared__ __align__(16) uint8_t lds[BYTES];
  __shared__ int rows[U];
  const int sub = DIRECT ? 1 : g.R.unit_rows / U;
  int e;
  const int count = find_unit<U, DIRECT>(g, blockIdx.y / sub, blockIdx.y % sub * U, &e, rows);
  if (count <= 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const int lr = lane >> 3, lk = lane & 7;                    // loads: row of eight, chunk of its line
  const int64_t len = TRANS ? g.N : g.K;
  const int steps = (int)((len + 63) / 64), waves = NW * g.splits, wi = (int)blockIdx.x * NW + wave;
  const int s0 = (int)((int64_t)steps * wi / waves), s1 = (int)((int64_t)steps * (wi + 1) / waves);
  uint8_t* img = lds + wave * IMG;
  // rows of z, then (A) the rank's rows of A; rows past the last repeat it (their results are not kept)
  const uint16_t* zp[2 * TILES];
#pragma unroll
  for (int i = 0; i < 2 * TILES; ++i) {
    const int r = 8 * i + lr;
    if (i < 2 * T) zp[i] = g.z + (int64_t)rows[min(r, count - 1)] * len + 8 * lk;
    else zp[i] = g.a + ((int64_t)e * g.rank + min(r - U, g.rank - 1)) * len + 8 * lk;
  }
  // B, transposed: lane c supplies rank column RB c + i to MFMA i
  const uint16_t* bp = TRANS ? g.b + ((int64_t)e * g.N + 8 * q) * g.rank + RB * c : nullptr;
  const int in_rank = RB * c < g.rank ? 8 : 0;
  f32x4_t acc[T][RB];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int i = 0; i < RB; ++i) acc[t][i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  u32x4_t next[2 * TILES];
  Cols8<TRANS ? RB : 1> bn[2];
  auto load = [&](int s) __attribute__((always_inline)) {
    const int64_t at = 64 * (int64_t)s;
    const bool whole = !TRANS || at + 64 <= len;
#pragma unroll
    for (int i = 0; i < 2 * TILES; ++i) {
      if (whole) next[i] = TRANS ? ld8(zp[i] + at) : ld16(zp[i] + at);
      else next[i] = at + 8 * lk < len ? ld8_tail(zp[i] - 8 * lk, at + 8 * lk, len) : (u32x4_t){0u, 0u, 0u, 0u};
    }
    if constexpr (TRANS) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t left = len - (at + 32 * j + 8 * q);
        bn[j].load(bp + (at + 32 * j) * g.rank, g.rank, whole ? in_rank : (int)max(min(left, (int64_t)in_rank), (int64_t)0));
      }
    }
  };
  if (s0 < s1) load(s0);
  for (int s = s0; s < s1; ++s) {
#pragma unroll
    for (int i = 0; i < 2 * TILES; ++i) st16(img + chunk_at(8 * i + lr, lk), next[i]);
    Cols8<TRANS ? RB : 1> bv[2];
    if constexpr (TRANS) {
      bv[0] = bn[0];
      bv[1] = bn[1];
    }
    __asm__ volatile("" ::: "memory");                        // a wave's LDS accesses stay in order
    if (s + 1 < s1) load(s + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      u32x4_t zv[T];
#pragma unroll
      for (int t = 0; t < T; ++t) zv[t] = ld16(img + chunk_at(16 * t + c, 4 * j + q));
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const u32x4_t a = TRANS ? bv[j].operand(TRANS ? i : 0) : ld16(img + chunk_at(U + 16 * i + c, 4 * j + q));
#pragma unroll
        for (int t = 0; t < T; ++t) acc[t][i] = mfma_bf16(a, zv[t], acc[t][i]);
      }
    }
    __asm__ volatile("" ::: "memory");
  }
  __syncthreads();                                            // the images give way to the sums
  float(*red)[U][LD] = reinterpret_cast<float(*)[U][LD]>(lds);
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
// their rows 16 at a time.  Lane c supplies column 4 c + b to MFMA b and so
// ends up with columns 4 c .. 4 c + 3 of rows 4 q + v: sixteen lanes read base
// and write y 128 consecutive bytes at a time (with the rows along the lanes
// instead, 16 bytes each, the address unit bound the kernel: m = 8192, n =
// 14336, rank 64 132 us).  Blocks go round the XCDs one by one, so block id i takes columns i % 8 + 8 k: each XCD sees
// an eighth of B_e, which stays in its L2 from group to group.
template <int RP, int T, bool DIRECT, bool TRANS>
__global__ void __launch_bounds__(256) k_lora_expand(LoraArgs g) {
  constexpr int S = RP == 16 ? 1 : RP / 16, HALF = RP == 16 ? 1 : RP / 32, U = 16 * T, LDH = 2 * RP + 8;
  __shared__ __align__(16) uint16_t hs[2][U][LDH];            // a row's h: RP values hi, RP values lo
  __shared__ __align__(16) int rows[2][U];
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
  const int64_t n0 = c0 + 64 * wave, n = n0 + 4 * c;          // the wave's and the lane's first column
  // rank column of MFMA step s (of 32 over [hi | lo]) that quarter q supplies first; RP = 16: one step, 0-1 hi, 2-3 lo
  auto rank0 = [q](int s) { return RP == 16 ? 8 * (q & 1) : 32 * s + 8 * q; };
  u32x4_t bv[TRANS ? 1 : 4][HALF];
  u32x2_t yv[T][4];
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
          const uint16_t* A = g.a + (int64_t)e * g.rank * g.K + n0 + 4 * c;
#pragma unroll
          for (int s = 0; s < HALF; ++s) cv[s].load(A + (int64_t)rank0(s) * g.K, g.K, rank0(s) < g.rank ? 8 : 0);
        } else {
          const uint16_t* B = g.b + (int64_t)e * g.N * g.rank;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int64_t nb = min(n + b, N - 1);
#pragma unroll
            for (int s = 0; s < HALF; ++s) {
              bv[b][s] = (u32x4_t){0u, 0u, 0u, 0u};
              if (rank0(s) < g.rank) bv[b][s] = ld16(B + nb * g.rank + rank0(s));
            }
          }
        }
      }
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int4 m4 = *reinterpret_cast<const int4*>(rw + 16 * t + 4 * q);
        const int m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          yv[t][v] = (u32x2_t){0u, 0u};
          if (g.base && 16 * t + 4 * q + v < count && n < N) yv[t][v] = ld4_tail(g.base + (int64_t)m[v] * N, n, N);
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
          acc[b] = mfma_bf16(hf[s], a, acc[b]);
        }
      }
      const int4 m4 = *reinterpret_cast<const int4*>(rw + 16 * t + 4 * q);
      const int m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if (16 * t + 4 * q + v >= count || n >= N) continue;
        u32x2_t o;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          o[k] = pack_bf16(lo_bf16(yv[t][v][k]) + acc[2 * k][v], hi_bf16(yv[t][v][k]) + acc[2 * k + 1][v]);
        st4_tail(g.y + (int64_t)m[v] * N, n, N, o);
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
  const dim3 block(64u * (unsigned)shrink_waves(RP, t));
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
