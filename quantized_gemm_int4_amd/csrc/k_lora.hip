// Low-rank adapters of many requests beside a shared projection.  For every
// row m of adapter e = ids[m]:
//   forward    h[m] = s_e A_e x[m]           y[m] = base[m] + B_e h[m]
//   gradient   g[m] = s_e B_e^T dy[m]        dx[m] = dx_base[m] + A_e^T g[m]
// that is, one contraction of long rows to the rank ("shrink") and one
// product back ("expand"), the gradient's with the transposed matrices
// (TRANS).  Rows are grouped by adapter into units that share the loads of
// their adapter's matrices.  Both products run on the bf16 MFMA; the rank is
// far too small for either to be bound by it: the shrink reads its rows once,
// the expand reads base and writes y once, and calls of few rows read the
// adapters.  An MFMA operand wants eight
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
// A row's place within 1024 rows is its rank among its wave's equal ids, by
// matching ballots, after the counts of the waves before.
__global__ void __launch_bounds__(kSortThreads)
k_lora_plan(const int32_t* __restrict__ ids, int64_t M, int L, int64_t C, int U, int64_t max_units,
            int32_t* __restrict__ units, int32_t* __restrict__ rows, int32_t* __restrict__ firsts) {
  __shared__ int hist[kSortWaves][512];
  __shared__ int before[512], after[512], base[512], uend[512];
  __shared__ int wsum[8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t lo = (int64_t)blockIdx.x * C, hi = min(lo + C, M);       // C is a multiple of kSortThreads
  int own = lo + tid < hi ? ids[lo + tid] : -1;
  for (int i = tid; i < 512; i += kSortThreads) before[i] = after[i] = 0;
  for (int i = tid; i < kSortWaves * 512; i += kSortThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  for (int64_t p0 = 0; p0 < M; p0 += 8 * kSortThreads) {
    int id[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t p = p0 + i * kSortThreads + tid;
      id[i] = p < M ? ids[p] : -1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int* cnt = p0 + i * kSortThreads < lo ? before : after;
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
  int nbits = 0;
  while ((1 << nbits) < L) ++nbits;
  const uint64_t lt = lane ? (~0ull >> (64 - lane)) : 0ull;
  for (int64_t p0 = lo; p0 < hi; p0 += kSortThreads) {
    const int e = own;
    const bool ok = e >= 0 && e < L;
    if (p0 + kSortThreads < hi) own = p0 + kSortThreads + tid < hi ? ids[p0 + kSortThreads + tid] : -1;
    uint64_t m = __ballot(ok);
    for (int bit = 0; bit < nbits; ++bit) {
      const uint64_t x = __ballot(ok && ((e >> bit) & 1));
      m &= ((e >> bit) & 1) ? x : ~x;
    }
    const int rank = __popcll(m & lt);
    if (ok && rank == 0) hist[wave][e] = __popcll(m);
    __syncthreads();
    int at = ok ? base[e] + rank : 0;
    if (ok)
      for (int w = 0; w < wave; ++w) at += hist[w][e];
    if (ok) rows[at] = (int32_t)(p0 + tid);
    if (p0 + kSortThreads >= hi) break;
    __syncthreads();
    if (ok && rank == 0) {
      atomicAdd(&base[e], __popcll(m));
      hist[wave][e] = 0;
    }
    __syncthreads();
  }
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
    // the unit's slots are read with its head, not after it; those behind its count are not used
    if (threadIdx.x < U) rows[threadIdx.x] = g.R.rows[(int64_t)u * g.R.unit_rows + first + threadIdx.x];
    *e = g.R.units[2 * u];
    const int count = min(g.R.units[2 * u + 1] - first, U);
    __syncthreads();
    return count;
  }
}

// 64 columns of B (rows of `rank` values, contiguous) through a wave's LDS
// image: whole lines are loaded and each MFMA's operand (lane (c, q): column 4
// c + b, rank values 32 s + 8 q ..) is read back from there.  Column 4 c + b
// has slot 16 b + c, whose 16-byte parts are rotated so that sixteen lanes'
// reads spread over the banks.
template <int RP> struct BGroup {
  static constexpr int P = RP / 8, BYTES = 64 * RP * 2;
  u32x4_t v[P];
  __device__ __forceinline__ void load(const uint16_t* B, int64_t n0, int64_t N, int rank, int lane) {
    const int per = rank / 8;
    const int64_t last = N * per - 1;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (i < per) v[i] = ld16(B + 8 * min(n0 * per + i * 64 + lane, last));
  }
  __device__ static int place(int slot, int part) { return (slot * P + ((part + slot * P / 16) & (P - 1))) * 16; }
  __device__ __forceinline__ void store(uint8_t* img, int rank, int lane) const {
    const int per = rank / 8;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (i < per) {
        const int ch = i * 64 + lane, col = ch / per;
        st16(img + place(16 * (col & 3) + (col >> 2), ch - col * per), v[i]);
      }
    __asm__ volatile("" ::: "memory");                        // a wave's LDS accesses stay in order
  }
  // part: r0 / 8 of the operand's first rank value
  __device__ __forceinline__ static u32x4_t operand(const uint8_t* img, int b, int c, int part, int rank) {
    return 8 * part < rank ? ld16(img + place(16 * b + c, part)) : (u32x4_t){0u, 0u, 0u, 0u};
  }
};


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
// no block barrier.  Now 26 us, of which reading x at the copy rate takes 13;
// dy with n = 14336, rank 32: 41 us, 5.7 TB/s.
template <int RP, int T, bool DIRECT, bool TRANS, int NW>
__global__ void __launch_bounds__(64 * NW) k_lora_shrink(LoraArgs g) {
  constexpr int RB = RP / 16, LD = RP + 4, U = 16 * T;
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
  auto load = [&](int s) __attribute__((always_inline)) {
    const int64_t at = 64 * (int64_t)s;
    const bool whole = !TRANS || at + 64 <= len;
#pragma unroll
    for (int i = 0; i < 2 * TILES; ++i) {
      if (whole) next[i] = TRANS ? ld8(zp[i] + at) : ld16(zp[i] + at);
      else next[i] = at + 8 * lk < len ? ld8_tail(zp[i] - 8 * lk, at + 8 * lk, len) : (u32x4_t){0u, 0u, 0u, 0u};
    }
  };
  // B's operands of half a step, loaded half a step ahead
  Cols8<TRANS ? RB : 1> bv[2];
  auto load_b = [&](int s, int j) __attribute__((always_inline)) {
    const int64_t at = 64 * (int64_t)s + 32 * j, left = len - (at + 8 * q);
    bv[j].load(bp + at * g.rank, g.rank, at + 32 <= len ? in_rank : (int)max(min(left, (int64_t)in_rank), (int64_t)0));
  };
  if (s0 < s1) {
    load(s0);
    if constexpr (TRANS) load_b(s0, 0);
  }
  for (int s = s0; s < s1; ++s) {
#pragma unroll
    for (int i = 0; i < 2 * TILES; ++i) st16(img + chunk_at(8 * i + lr, lk), next[i]);
    __asm__ volatile("" ::: "memory");                        // a wave's LDS accesses stay in order
    if (s + 1 < s1) load(s + 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (TRANS) {
        if (j == 0) load_b(s, 1);
        else if (s + 1 < s1) load_b(s + 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
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

// Those of rows m0 .. m0 + 63 that have no adapter, columns [c0, c1); a block
// of 256 threads.  list: 64 ints of LDS.  Eight rows of 256 columns at a time,
// two loads in flight a thread.
__device__ __forceinline__ void copy_rest(const LoraArgs& g, int64_t m0, int64_t n, int64_t c0, int64_t c1, bool zero_h,
                                          int* list) {
  const int lane = threadIdx.x & 63;
  const bool in = m0 + lane < g.M;
  const int e = in ? g.ids[m0 + lane] : 0;
  const bool none = in && (e < 0 || e >= g.L);
  const uint64_t m = __ballot(none);
  const int count = __popcll(m);
  if (count == 0) return;
  if (threadIdx.x < 64 && none) list[__popcll(m & (lane ? (~0ull >> (64 - lane)) : 0ull))] = lane;
  __syncthreads();
  if (g.base != g.y)
    for (int64_t cb = c0 + 8 * (threadIdx.x & 31); cb < c1; cb += 256)
      for (int i = threadIdx.x >> 5; i < count; i += 16) {
        u32x4_t v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          v[k] = (u32x4_t){0u, 0u, 0u, 0u};
          if (g.base && i + 8 * k < count) v[k] = ld8_tail(g.base + (m0 + list[i + 8 * k]) * n, cb, n);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (i + 8 * k < count) st8_tail(g.y + (m0 + list[i + 8 * k]) * n, cb, n, v[k]);
      }
  if (zero_h)
    for (int i = threadIdx.x; i < count * g.rank; i += 256) g.h[(m0 + list[i / g.rank]) * g.rank + i % g.rank] = 0.f;
}

// One block per (cols columns, group of units, or 64 rows of which those
// without an adapter are copied): y = base + B_e h.  A wave holds 64 columns
// of B_e in registers while its group's units have the same adapter and takes
// their rows 16 at a time.  Lane c supplies column 4 c + b to MFMA b and so
// ends up with columns 4 c .. 4 c + 3 of rows 4 q + v: sixteen lanes read base
// and write y 128 consecutive bytes at a time (with the rows along the lanes
// instead, 16 bytes each, the address unit bound the kernel: m = 8192, n =
// 14336, rank 64 132 us; now 112 us, 4.2 TB/s of base and y).  Blocks go round
// the XCDs one by one, so block id i takes its columns from the eighth i % 8:
// each XCD sees an eighth of B_e, which stays in its L2 from group to group,
// and writes neighbouring parts of a row.
// A row of h in LDS: RP values of each term; RP = 16 has the fourth too, so
// that two MFMAs of 32 take the row.
constexpr int h_values(int rp) { return rp == 16 ? 64 : kTerms * rp; }
template <int RP, int T> struct ExpandLds {
  static constexpr int U = 16 * T;
  __align__(16) uint16_t hs[U][h_values(RP) + 8];             // one image: find_unit's barrier comes before the next unit's
  __align__(16) int rows[2][U < 32 ? 32 : U];                 // 64 in all: copy_rest's list
};
template <int RP, int T, bool DIRECT, bool TRANS>
__device__ __forceinline__ void expand_block(const LoraArgs& g, uint32_t block, ExpandLds<RP, T>& lds) {
  constexpr int S = h_values(RP) / 32, HALF = RP == 16 ? 1 : RP / 32, U = 16 * T;
  auto& hu = lds.hs;
  auto& rows = lds.rows;
  const int64_t N = TRANS ? g.K : g.N;
  const int per = (int)((N + 8 * g.cols - 1) / (8 * g.cols));             // column slabs per XCD
  const uint32_t id = block >> 3;
  const int gi = (int)(id / per), slab = (int)(block & 7) * per + (int)(id % per);
  const int64_t c0 = (int64_t)slab * g.cols, c1 = min(c0 + g.cols, N);
  if (c0 >= N) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const bool keep = !TRANS && g.h && slab == 0;
  const int groups = DIRECT ? (int)g.M : (int)((g.R.max_units + g.group - 1) / g.group);
  if (!DIRECT && gi >= groups) {
    copy_rest(g, (int64_t)(gi - groups) * 64, N, c0, c1, keep, rows[0]);
    return;
  }
  // rank column of MFMA step s (of 32 over the terms) that quarter q supplies first; RP = 16: two terms a step
  auto rank0 = [q](int s) { return RP == 16 ? 8 * (q & 1) : 32 * s + 8 * q; };
  u32x4_t bv[TRANS ? 1 : 4][HALF];
  u32x2_t yv[T][4];
  Cols8<4> cv[TRANS ? HALF : 1];
  int have = -1;
  const int u0 = DIRECT ? gi : gi * g.group, un = DIRECT ? gi + 1 : (int)min((int64_t)u0 + g.group, g.R.max_units);
  for (int u = u0; u < un; ++u) {
    int e, *rw = rows[u & 1];
    const int count = find_unit<U, DIRECT>(g, u, 0, &e, rw);
    if (count <= 0) {
      if (DIRECT && count < 0 && wave == 0) copy_row(g, u, N, c0, c1, keep);
      return;                                                 // units behind the last used one are empty too
    }
    int64_t n0 = c0 + 64 * wave, n = n0 + 4 * c;              // the wave's and the lane's first column
    auto load_group = [&]() __attribute__((always_inline)) {
      if (e != have || T < 4) {
        have = e;
        if constexpr (TRANS) {
          const uint16_t* A = g.a + (int64_t)e * g.rank * g.K + n;
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
    };
    if (n0 < c1) load_group();
    loads_first();
    // h of the unit's rows: the splits' sums in split order, as bf16 terms
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
        uint32_t t[2][4];
        split4(v[0], v[1], t[0]);
        split4(v[2], v[3], t[1]);
#pragma unroll
        for (int k = 0; k < h_values(RP) / RP; ++k)
          *reinterpret_cast<u32x2_t*>(&hu[row][RP * k + r0]) = (u32x2_t){t[0][k], t[1][k]};
      }
    };
    if (g.splits == 1) stage(Int<1>{});
    else if (lora_max_splits(RP, U, TRANS) == 4 || g.splits <= 4) stage(Int<4>{});
    else stage(Int<8>{});
    __syncthreads();
    while (n0 < c1) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if (16 * t >= count) break;
      const uint16_t* hr = hu[min(16 * t + c, count - 1)] + 8 * q;
      f32x4_t acc[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[b] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s0 = 0; s0 < HALF; ++s0) {
        u32x4_t hf[S / HALF];
#pragma unroll
        for (int i = 0; i < S / HALF; ++i) hf[i] = ld16(hr + 32 * (s0 + HALF * i));
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          u32x4_t a;
          if constexpr (TRANS) a = cv[s0].operand(b);
          else a = bv[b][s0];
#pragma unroll
          for (int i = 0; i < S / HALF; ++i) acc[b] = mfma_bf16(hf[i], a, acc[b]);
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
      if constexpr (T == 4) break;                            // one part of the columns, several units
      n0 += kLoraCols;
      n += kLoraCols;
      if (n0 < c1) load_group();
    }
  }
}

template <int RP, int T, bool DIRECT>
__global__ void __launch_bounds__(256) k_lora_expand(LoraArgs g) {
  __shared__ ExpandLds<RP, T> lds;
  expand_block<RP, T, DIRECT, false>(g, blockIdx.x, lds);
}

// g (the splits' sums) or, is_h, h of 32 of a unit's rows
// in the order of the outer product's operands, so that a wave loads each
// with one contiguous access: [32-row step][term][16-rank block][lane][8],
// lane (c, q) holding rank 16 k + c of rows 32 s + 8 q .. + 7; zeros beyond
// the rank and the unit's rows.
template <int RP>
__device__ __forceinline__ void pack_block(const LoraGradArgs& g, int u, bool is_h, int half, float (*v)[RP + 1]) {
  constexpr int MS = lora_max_splits(RP, kLoraUnit, true);
  const int count = g.R.units[2 * u + 1] - 32 * half;
  if (count <= 0) return;                                     // unused units and steps are not read
  const int32_t* rows = g.R.rows + (int64_t)u * kLoraUnit + 32 * half;
  const float* src = is_h ? g.h : g.part;
  const int splits = is_h ? 1 : g.splits;
#pragma unroll
  for (int i0 = 0; i0 < 32 * (RP / 4); i0 += 256) {
    const int i = i0 + threadIdx.x, row = i / (RP / 4), r = 4 * (i % (RP / 4));
    if (i >= 32 * (RP / 4)) break;
    f32x4_t s = {0.f, 0.f, 0.f, 0.f}, p[MS];
    if (row < count && r < g.rank) {
      const int64_t at = (int64_t)rows[row] * g.rank + r;
#pragma unroll
      for (int k = 0; k < MS; ++k)
        p[k] = *reinterpret_cast<const f32x4_t*>(src + (int64_t)min(k, splits - 1) * g.M * g.rank + at);
      loads_first();
#pragma unroll
      for (int k = 0; k < MS; ++k)
        if (k < splits) s += p[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[row][r + k] = s[k];
  }
  __syncthreads();
  uint16_t* out = (is_h ? g.ht : g.gt) + ((int64_t)u * 2 + half) * kTerms * RP * 32;
  for (int i = threadIdx.x; i < RP * 4; i += 256) {
    const int lane = i & 63, k = i >> 6, r = 16 * k + (lane & 15), m = 8 * (lane >> 4);
    uint32_t t[4][4];
#pragma unroll
    for (int p = 0; p < 4; ++p) split4(v[m + 2 * p][r], v[m + 2 * p + 1][r], t[p]);
#pragma unroll
    for (int j = 0; j < kTerms; ++j) st16(out + RP * 32 * j + 8 * i, (u32x4_t){t[0][j], t[1][j], t[2][j], t[3][j]});
  }
}

// Zeros for da and db of an adapter without rows; block `part` of `parts`.
__device__ __forceinline__ void zero_block(const LoraGradArgs& g, int e, int part, int parts) {
  if (g.M && g.R.first[e] != g.R.first[e + 1]) return;
  const int64_t na = (int64_t)g.rank * g.K, nb = (int64_t)g.rank * g.N;
  for (int64_t at = 8 * ((int64_t)part * 256 + threadIdx.x); at < na + nb; at += 2048 * (int64_t)parts)
    st16(at < na ? g.da + e * na + at : g.db + e * nb + at - na, (u32x4_t){0u, 0u, 0u, 0u});
}

// What the gradient can do once g is there, in one launch: the packed g and h
// (blocks [0, packs)), the zeros (zeros blocks), and dx = dx_base + A^T g
// (m = 777, k = 2048, rank 16: 7.6 us against 7.2 + 3.0 in two launches; m =
// 8192, k = 4096, rank 32: 31 us, 4.3 TB/s of dx_base and dx).
template <int RP>
__global__ void __launch_bounds__(256, 2) k_lora_dx(LoraArgs g, LoraGradArgs o, int packs, int zero_parts, int zeros) {
  __shared__ ExpandLds<RP, 4> lds;
  static_assert(sizeof(lds.hs) >= 32 * (RP + 1) * sizeof(float), "the packing pass fits the expansion's LDS");
  const int b = (int)blockIdx.x;
  if (b < packs) {
    if (b >> 2 < o.R.max_units) pack_block<RP>(o, b >> 2, b & 1, (b >> 1) & 1, reinterpret_cast<float(*)[RP + 1]>(&lds.hs));
  } else if (b < packs + zeros) {
    const int z = b - packs;
    if (z / zero_parts < o.L) zero_block(o, z / zero_parts, z % zero_parts, zero_parts);
  } else {
    expand_block<RP, 4, false, true>(g, (uint32_t)(b - packs - zeros), lds);
  }
}

// Both products of a call of few rows in one launch: every block contracts
// its unit's rows over all of K by itself and expands a part of the columns.
// A is read once per part, from the L2 after the first, which costs less than
// a second launch and the round trips at its start while A is small.
// grid (column parts, rows); NW waves.
constexpr int small_waves(int rp) { return rp == 64 ? 8 : 16; }
template <int RP>
__global__ void __launch_bounds__(64 * small_waves(RP)) k_lora_small(LoraArgs g) {
  constexpr int RB = RP / 16, NW = small_waves(RP), LD = RP + 4, S = h_values(RP) / 32, HALF = RP == 16 ? 1 : RP / 32;
  constexpr int NB = RB == 1 ? 4 : 2, IMG = (1 + RB) * 2048, LDH = h_values(RP) + 8;
  constexpr int BYTES = NW * IMG > NW * 16 * LD * 4 ? NW * IMG : NW * 16 * LD * 4;
  __shared__ __align__(16) uint8_t lds[BYTES];
  __shared__ __align__(16) uint16_t hs[16][LDH];
  __shared__ __align__(16) int rows[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
  const int64_t N = g.N, K = g.K;
  const int64_t groups = (N + 63) / 64, g0 = groups * blockIdx.x / gridDim.x, g1 = groups * (blockIdx.x + 1) / gridDim.x;
  const bool keep = g.h && blockIdx.x == 0;
  int e;
  const int count = find_unit<16, true>(g, blockIdx.y, 0, &e, rows);
  if (count <= 0) {
    if (count < 0 && wave == 0) copy_row(g, blockIdx.y, N, 64 * g0, min(64 * g1, N), keep);
    return;
  }
  auto rank0 = [q](int s) { return RP == 16 ? 8 * (q & 1) : 32 * s + 8 * q; };
  const uint16_t* B = g.b + (int64_t)e * N * g.rank;
  const int4 m4 = *reinterpret_cast<const int4*>(rows + 4 * q);
  const int m[4] = {m4.x, m4.y, m4.z, m4.w};
  BGroup<RP> bg;
  u32x2_t yv[4];
  auto load_group = [&](int64_t n0) __attribute__((always_inline)) {
    const int64_t n = n0 + 4 * c;
    bg.load(B, n0, N, g.rank, lane);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      yv[v] = (u32x2_t){0u, 0u};
      if (g.base && 4 * q + v < count && n < N) yv[v] = ld4_tail(g.base + (int64_t)m[v] * N, n, N);
    }
  };
  // h: the waves split K into steps of 64, NB steps' loads in flight
  const int steps = (int)(K / 64), s0 = steps * wave / NW, s1 = steps * (wave + 1) / NW;
  uint8_t* img = lds + wave * IMG;
  const int lr = lane >> 3, lk = lane & 7;
  const uint16_t* zp[2 * (1 + RB)];
#pragma unroll
  for (int i = 0; i < 2 * (1 + RB); ++i) {
    const int r = 8 * i + lr;
    zp[i] = i < 2 ? g.z + (int64_t)rows[min(r, count - 1)] * K + 8 * lk
                  : g.a + ((int64_t)e * g.rank + min(r - 16, g.rank - 1)) * K + 8 * lk;
  }
  f32x4_t acc[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) acc[i] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  if (g0 + wave < g1) load_group(64 * (g0 + wave));
  for (int s = s0; s < s1; s += NB) {
    u32x4_t v[NB][2 * (1 + RB)];
#pragma unroll
    for (int j = 0; j < NB; ++j)
      if (s + j < s1)
#pragma unroll
        for (int i = 0; i < 2 * (1 + RB); ++i)
          if (i != 1 || count > 8) v[j][i] = ld16(zp[i] + 64 * (s + j));
    loads_first();
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if (s + j >= s1) break;
#pragma unroll
      for (int i = 0; i < 2 * (1 + RB); ++i)
        if (i != 1 || count > 8) st16(img + chunk_at(8 * i + lr, lk), v[j][i]);
      __asm__ volatile("" ::: "memory");
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4_t zv = ld16(img + chunk_at(min(c, count - 1), 4 * h + q));
#pragma unroll
        for (int i = 0; i < RB; ++i)
          acc[i] = mfma_bf16(ld16(img + chunk_at(16 + 16 * i + c, 4 * h + q)), zv, acc[i]);
      }
      __asm__ volatile("" ::: "memory");
    }
  }
  __syncthreads();                                            // the images give way to the sums
  float(*red)[16][LD] = reinterpret_cast<float(*)[16][LD]>(lds);
#pragma unroll
  for (int i = 0; i < RB; ++i) *reinterpret_cast<f32x4_t*>(&red[wave][c][16 * i + 4 * q]) = acc[i];
  __syncthreads();
  const float sc = g.scales[e];
  for (int i = threadIdx.x; i < count * (RP / 2); i += 64 * NW) {
    const int row = i / (RP / 2), r = 2 * (i % (RP / 2));
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      a += red[w][row][r];
      b += red[w][row][r + 1];
    }
    a = r < g.rank ? a * sc : 0.f;
    b = r < g.rank ? b * sc : 0.f;
    if (keep && r < g.rank) {
      g.h[(int64_t)rows[row] * g.rank + r] = a;
      g.h[(int64_t)rows[row] * g.rank + r + 1] = b;
    }
    uint32_t t[4];
    split4(a, b, t);
#pragma unroll
    for (int k = 0; k < h_values(RP) / RP; ++k) *reinterpret_cast<uint32_t*>(&hs[row][RP * k + r]) = t[k];
  }
  __syncthreads();
  u32x4_t hf[S];
#pragma unroll
  for (int s = 0; s < S; ++s) hf[s] = ld16(&hs[min(c, count - 1)][32 * s + 8 * q]);
  for (int64_t gi = g0 + wave; gi < g1; gi += NW) {
    const int64_t n = 64 * gi + 4 * c;
    bg.store(img, g.rank, lane);
    f32x4_t o[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      o[b] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < S; ++s)
        o[b] = mfma_bf16(hf[s], BGroup<RP>::operand(img, b, c, rank0(s % HALF) / 8, g.rank), o[b]);
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (4 * q + v >= count || n >= N) continue;
      u32x2_t w;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        w[k] = pack_bf16(lo_bf16(yv[v][k]) + o[2 * k][v], hi_bf16(yv[v][k]) + o[2 * k + 1][v]);
      st4_tail(g.y + (int64_t)m[v] * N, n, N, w);
    }
    __asm__ volatile("" ::: "memory");
    if (gi + NW < g1) load_group(64 * (gi + NW));
  }
}

hipError_t launch_lora_small(const LoraArgs& g, int parts, hipStream_t st) {
  const dim3 grid((unsigned)parts, (unsigned)g.M);
  switch (lora_rp(g.rank)) {
    case 16: hipLaunchKernelGGL(k_lora_small<16>, grid, dim3(64 * small_waves(16)), 0, st, g); break;
    case 32: hipLaunchKernelGGL(k_lora_small<32>, grid, dim3(64 * small_waves(32)), 0, st, g); break;
    case 64: hipLaunchKernelGGL(k_lora_small<64>, grid, dim3(64 * small_waves(64)), 0, st, g); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
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
  constexpr int W1 = lora_waves(RP, 16, false), W2 = lora_waves(RP, 64, TRANS);
  if constexpr (!TRANS) {
    if (direct) hipLaunchKernelGGL((k_lora_shrink<RP, 1, true, false, W1>), grid, dim3(64 * W1), 0, st, g);
    else if (t == 1) hipLaunchKernelGGL((k_lora_shrink<RP, 1, false, false, W1>), grid, dim3(64 * W1), 0, st, g);
  }
  if (t == 2) hipLaunchKernelGGL((k_lora_shrink<RP, 2, false, TRANS, W2>), grid, dim3(64 * W2), 0, st, g);
}

// blocks of the expansion, a multiple of 8
static int64_t expand_grid(const LoraArgs& g, int64_t columns, bool direct, bool rest) {
  const int64_t per = (columns + 8 * g.cols - 1) / (8 * g.cols);
  return 8 * per * (direct ? g.M : (g.R.max_units + g.group - 1) / g.group + (rest ? (g.M + 63) / 64 : 0));
}

template <int RP>
static void run_expand(const LoraArgs& g, bool direct, hipStream_t st) {
  const dim3 grid((unsigned)expand_grid(g, g.N, direct, g.base != g.y || g.h));
  if (direct) hipLaunchKernelGGL((k_lora_expand<RP, 1, true>), grid, dim3(256), 0, st, g);
  else if (g.R.unit_rows == 16) hipLaunchKernelGGL((k_lora_expand<RP, 1, false>), grid, dim3(256), 0, st, g);
  else if (g.R.unit_rows == 32) hipLaunchKernelGGL((k_lora_expand<RP, 2, false>), grid, dim3(256), 0, st, g);
  else hipLaunchKernelGGL((k_lora_expand<RP, 4, false>), grid, dim3(256), 0, st, g);
}

hipError_t launch_lora_dx(const LoraArgs& g, const LoraGradArgs& o, hipStream_t st) {
  const int packs = (int)((4 * o.R.max_units + 7) / 8 * 8);
  const int zero_parts = lora_zero_parts(o.rank, o.K, o.N);
  const int zeros = (o.L * zero_parts + 7) / 8 * 8;           // block ids of the expansion keep their XCDs
  const dim3 grid((unsigned)(packs + zeros + (g.y ? expand_grid(g, g.K, false, g.base != g.y) : 0)));
  switch (lora_rp(o.rank)) {
    case 16: hipLaunchKernelGGL(k_lora_dx<16>, grid, dim3(256), 0, st, g, o, packs, zero_parts, zeros); break;
    case 32: hipLaunchKernelGGL(k_lora_dx<32>, grid, dim3(256), 0, st, g, o, packs, zero_parts, zeros); break;
    case 64: hipLaunchKernelGGL(k_lora_dx<64>, grid, dim3(256), 0, st, g, o, packs, zero_parts, zeros); break;
    default: hipLaunchKernelGGL(k_lora_dx<128>, grid, dim3(256), 0, st, g, o, packs, zero_parts, zeros);
  }
  return hipGetLastError();
}

hipError_t launch_lora_expand(const LoraArgs& g, bool direct, hipStream_t st) {
  switch (lora_rp(g.rank)) {
    case 16: run_expand<16>(g, direct, st); break;
    case 32: run_expand<32>(g, direct, st); break;
    case 64: run_expand<64>(g, direct, st); break;
    default: run_expand<128>(g, direct, st);
  }
  return hipGetLastError();
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

}  // namespace hm
