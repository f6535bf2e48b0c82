// Products of 8-bit integer layers and of their gradients, 128 x 128 output
// tiles: O[q][p] = sum_c Q[q][c] P[p][c] on 32x32 MFMAs, int8 codes with exact
// integer sums (32x32x32) or bf16 with fp32 sums (32x32x16).
//
// A block of four waves, one a SIMD, each with 64 x 64 of the tile.  The MFMA's
// rows are the output's columns p, so that a lane holds four neighbouring
// columns of one output row.  Operands come through LDS in steps of 128 bytes
// of the contraction by 16-byte direct buffer-to-LDS copies; reads past an
// array give zeros, so no size has to be padded.  Gradients of few tiles read
// their int8 operand (weights for dx, rows of x for dw) as it is and turn it into bf16
// between the MFMAs (a step of 0.66 us for 0.51 on a full card, but no bf16 copy of the operand to make
// first: m = 128, n = 14336, k = 4096 dx 33 us for 63; m = 1024 161 for 145).  During step s its operands are
// in registers, those of step s + 1 are read from LDS between the MFMAs, and ST
// stages hold steps s + 1 .. s + ST, so that a copy has ST - 1 steps to land.
//
// Where one round of tiles has the card, a block has a compute unit for itself and four
// stages, and a fifth wave touches later steps' lines (Ahead; product of m = 1021, n = 4099, k = 7168 58 us
// without it, 44 with): a step's 32 KiB take 0.22 us from L2 at the 64 bytes a clock that a compute unit gets, twice that with
// all of them at it.  A step is 0.46 to 0.54 us on 256 tiles of Gaussian codes (m = 1024, n = 4096, k = 1792 to 14336, calls in a row;
// of zeros, which draw less power, 0.40), for 512 cycles of MFMA, 0.21 us.  Counters of that product at k = 7168, one call at a time, at
// 2.35 GHz, as shares of the kernel's 85000 cycles: the path that brings lines from L2 into LDS 65 % busy, and
// waiting for L2 in 26 %; matrix cores 34 %; LDS reads 18 %, no bank conflicts.  So copies, not LDS, keep the matrix
// cores waiting, and power comes second.  Where more tiles follow, two blocks with two stages each share one, so that
// the start and the end of one (4 us) go with the other's steps: product m = 4313, n = 5402, k = 256 20.1 us
// for 30.7 with four stages, m = 755, n = 9616, k = 6272 51.6 for 59.3, dw m = 359, n = 1600, k = 5504 17.1 for 22.2; but 220 tiles of
// k = 5632 32.8 for 28.5.  Against the 256 x 256 tiles: m = 4313 as above 28.6 us, m = 1364, n = 20992, k = 3968 125.4 here for 113.8.
//
// Tiles that do not fill the card's 256 compute units in a last round (or all of
// them, where there are fewer) are split along the contraction: `cut` blocks a
// tile write their sums to the workspace and k_i8_finish adds them up in order.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "common.h"
#include "i8.h"
#include "i8_tile.h"

namespace hm {

namespace {

// How P is held: contracted along its rows, int8 codes whose rows are contracted, bf16 whose rows are.
enum PMode : int { P_ROWS, P_CODES, P_BF16 };
// P8: P is int8 codes whose rows are contracted (gradients); then a stage also has a slot of 64 scales for each wave
template <bool P8> constexpr int kP = P8 ? Codes::kBytes : kHalfBytes;
template <bool P8> constexpr int kStage = kP<P8> + kHalfBytes;             // P and Q of one step
template <bool P8, int ST> constexpr int kScales = ST * kStage<P8>;        // the slots, or the scales of 128 + 128 results
template <bool P8, int ST> constexpr int kTileLds = kScales<P8, ST> + (P8 ? ST * 1024 : 1024) + 256;   // (and what is touched)
constexpr int kAhead = 4, kStages = 4;             // steps between a touch and its copy, between a copy and its use

// The lines of step first + kStages + kAhead on, a step at each of the compute waves' barriers.
template <int PM, bool QS, int EPI>
__device__ void run_ahead(const TileArgs& a, int tp, int tq, int first, int steps, int tiles_p, int tiles_q, int lane, uint8_t* place) {
  const int qs = min(4, tiles_q - (tq & ~3)), ps = min(8, tiles_p);    // blocks on the same rows of P, of Q
  const int64_t from = first + kStages;
  constexpr int kQ = QS ? 2 : 1;
  Ahead p, u, q;
  if (PM == P_ROWS && kPairs<EPI>) {
    const int64_t at = (int64_t)tp * (kI8Tile / 2) * a.p_ld + from * 128;
    p.init(a.p, a.p_bytes, at, 128, a.p_ld, 64, 1, tq & 3, qs, lane);
    u.init(a.p + a.p_bytes, a.p_bytes, at, 128, a.p_ld, 64, 1, tq & 3, qs, lane);
  } else if (PM == P_ROWS) {
    p.init(a.p, a.p_bytes, (int64_t)tp * kI8Tile * a.p_ld + from * 128, 128, a.p_ld, 128, 1, tq & 3, qs, lane);
  } else {
    constexpr int kP = PM == P_BF16 ? 2 : 1;       // lines of a contracted row
    p.init(a.p, a.p_bytes, (int64_t)tp * kI8Tile * kP + from * 64 * a.p_ld, 64 * a.p_ld, a.p_ld, 64 * kP, kP, tq & 3, qs, lane);
  }
  if (QS) q.init(a.q, a.q_bytes, (int64_t)tq * kI8Tile * kQ + from * 64 * a.q_ld, 64 * a.q_ld, a.q_ld, 128, 2, tp % ps, ps, lane);
  else q.init(a.q, a.q_bytes, (int64_t)tq * kI8Tile * a.q_ld + from * 128, 128, a.q_ld, 128, 1, tp % ps, ps, lane);
  auto touch = [&](int s) __attribute__((always_inline)) {
    if (s >= steps) return;
    p.touch(place);
    if (PM == P_ROWS && kPairs<EPI>) u.touch(place);
    q.touch(place);
  };
  for (int s = 0; s < kAhead; ++s) touch(kStages + s);
  __asm__ volatile("s_barrier" ::: "memory");
  int s = 0;
  do {
    __asm__ volatile("s_barrier" ::: "memory");
    touch(s + kStages + kAhead);
    __asm__ volatile("s_barrier" ::: "memory");
    touch(s + 1 + kStages + kAhead);
    s += 2;
  } while (s < steps);
  __asm__ volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
}

template <class T, int PM, bool QS, int EPI, int ST>
__global__ void __launch_bounds__(ST == 4 ? 320 : 256, ST == 4 ? 1 : 2)
k_i8_tile(TileArgs a, TilePlan pl) {
  constexpr bool P8 = PM == P_CODES, PS = PM == P_BF16;
  // blocks of 32 of a wave: 2 x 2, codes 1 x 4 (no other wave converts the same ones)
  constexpr int PB = P8 ? 1 : 2, QB = P8 ? 4 : 2;
  using Acc = typename Mma<T>::Acc;
  extern __shared__ __align__(1024) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = P8 ? wave : wave & 1, wq = P8 ? 0 : wave >> 1;
  const int all = (int)((a.kbytes + 127) / 128);
  const uint32_t whole = 8 * ((uint32_t)(pl.full + 7) / 8);
  int tp, tq, first = 0, last = all, item = -1;
  if (blockIdx.x < whole) {
    if (!tile_of(pl.full, whole, 0, pl.tiles_p, pl.tiles_q, tp, tq)) return;
  } else {
    // the tiles of one part of the contraction after each other: neighbours share operands
    const uint32_t rest = (uint32_t)(pl.tiles_p * pl.tiles_q - pl.full), total = rest * pl.cut;
    const uint32_t j = number_of(total, blockIdx.x - whole, gridDim.x - whole, 0);
    if (j >= total) return;
    const uint32_t part = j / rest, t = j - part * rest;
    tile_at(pl.full + t, pl.tiles_p, pl.tiles_q, tp, tq);
    item = (int)(t * pl.cut + part);
    first = (int)part * pl.per;
    last = min(all, first + pl.per);
  }
  const int steps = last - first;
  float* sc = reinterpret_cast<float*>(lds + kScales<P8, ST>);
  if (std::is_same<T, int8_t>::value) {
    if (tid < kI8Tile) sc[tid] = a.ps[p_row<EPI>(a, tp, kI8Tile, tid)];
    else if (tid < 2 * kI8Tile) sc[tid] = a.qs[min((int64_t)tq * kI8Tile + tid - kI8Tile, a.rows - 1)];
  }
  if constexpr (ST == 4) {
    if (wave == 4) {
      run_ahead<PM, QS, EPI>(a, tp, tq, first, steps, pl.tiles_p, pl.tiles_q, lane, lds + kTileLds<P8, ST> - 256);
      return;
    }
  }
  Side<QS, false> Q;
  Q.init(a.q, a.q_ld, a.q_bytes, kI8Tile, lane, wave, a.kbytes);
  Q.tile(tq, first);
  Frags<QS, QB> fq;
  fq.init(lds + kP<P8>, lane, wq);
  std::conditional_t<P8, Codes, Side<PS, kPairs<EPI>>> P;
  Frags<PS> fp;
  uint8_t* const slot = lds + kScales<P8, ST> + wave * 256;
  if constexpr (P8) {
    P.init(a.p, a.p_ld, a.p_bytes, a.ps, a.terms, tp, first, lane, wave, lds, slot);
  } else {
    P.init(a.p, a.p_ld, a.p_bytes, kI8Tile, lane, wave, a.kbytes);
    P.tile(tp, first);
    fp.init(lds, lane, wp);
  }

  Acc acc[PB][QB];
#pragma unroll
  for (int i = 0; i < PB; ++i)
#pragma unroll
    for (int j = 0; j < QB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  // Copies of a step, i = 0..7 (codes: seven), into stage `at`; a step past the last copies zeros, so that the
  // waits can count on as many a step.
  auto begin = [&](int s) __attribute__((always_inline)) {
    if constexpr (P8) P.step(first + s, last);
    else P.step(first + s, last, all);
    Q.step(first + s, last, all);
  };
  auto copy = [&](int i, int at) __attribute__((always_inline)) {
    uint8_t* st = lds + at * kStage<P8>;
    if (i & 1) Q.copy(0, i >> 1, st + kP<P8>, wave);
    else if constexpr (!P8) P.copy(0, i >> 1, st, wave);
    else if (i < 6) P.copy(i >> 1, st, slot + at * 1024, wave);
  };
  constexpr int kCopies = P8 ? 7 : 8;
#pragma unroll
  for (int s = 0; s < ST; ++s) {
    begin(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) copy(i, s);
  }
  // Operands of a step in registers (codes as they are, with their scales).
  struct Ops {
    std::conditional_t<P8, u32x2_t, u32x4_t> p[PB][4];
    u32x4_t q[QB][4];
    f32x4_t s[4][2];
  };
  // part i = 0..15 of a step's operands, from a stage
  auto read = [&](Ops& o, int i, int stage) __attribute__((always_inline)) {
    const int ks = i >> 2, x = i & 3;
    const auto mq = fq.moved(stage * kStage<P8>);
    if constexpr (P8) {
      o.q[x][ks] = mq.read(0, x, ks);
      if (x == 0) o.p[0][ks] = P.read(stage * kStage<P8>, ks);
      else if (x < 3) o.s[ks][x - 1] = P.scales(stage * 1024, ks, x - 1);
    } else if (x < 2) {
      o.p[x][ks] = fp.moved(stage * kStage<P8>).read(0, x, ks);
      o.q[x][ks] = mq.read(0, x, ks);
    }
  };
  Ops a0, a1;
  __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((ST - 1) * kCopies) : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) read(a0, i, 0);
  // one step on operands o, while those of the next are read and step s + 4 is copied
  int at = 0;                                      // stage of step s
  auto step = [&](int s, const Ops& o, Ops& next) __attribute__((always_inline)) {
    const int after = (at + 1) & (ST - 1);
    begin(s + ST);
    // step s + 1 has landed (two steps' copies are newer), and all waves hold step s in registers
    __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((ST - 2) * kCopies) : "memory");
    u32x4_t v[2];                                  // codes: values of parts ks and ks + 1
    auto values = [&](int ks, int h) __attribute__((always_inline)) {
      if constexpr (P8) {
        const u32x2_t x = Codes::values(o.p[0][ks][h], o.s[ks][h]);
        v[ks & 1][2 * h] = x[0];
        v[ks & 1][2 * h + 1] = x[1];
      }
    };
    values(0, 0);
    values(0, 1);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int ks = i >> 2, x = P8 ? 0 : (i >> 1) & 1, y = P8 ? i & 3 : i & 1;
      if constexpr (P8) acc[x][y] = Mma<T>::run(v[ks & 1], o.q[y][ks], acc[x][y]);
      else acc[x][y] = Mma<T>::run(o.p[x][ks], o.q[y][ks], acc[x][y]);
      if (P8 || (i & 1)) read(next, P8 ? i : 4 * (i >> 2) + ((i >> 1) & 1), after);
      if ((i & 1) == 0) copy(i >> 1, at);
      if (P8 && (i & 1) && ks < 3) values(ks + 1, (i >> 1) & 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    at = after;
  };
  int s = 0;
  do {                                             // two steps a round; the second may be all zeros
    step(s, a0, a1);
    step(s + 1, a1, a0);
    s += 2;
  } while (s < steps);
  // the stages have been read by all waves, and no copy is in flight
  __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if (item >= 0) {
    // the sums as they are, [128 q][128 p] of this item
    auto* out = reinterpret_cast<typename Mma<T>::Sum*>(pl.part) + (int64_t)item * kI8Tile * kI8Tile;
#pragma unroll
    for (int x = 0; x < PB; ++x)
#pragma unroll
      for (int y = 0; y < QB; ++y)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u32x4_t v;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const typename Mma<T>::Sum one = acc[x][y][4 * j + e];
            v[e] = __builtin_bit_cast(uint32_t, one);
          }
          st16(out + (wq * 64 + y * 32 + (lane & 31)) * kI8Tile + wp * 32 * PB + x * 32 + 8 * j + 4 * (lane >> 5), v);
        }
    return;
  }
  const int64_t r0 = (int64_t)tq * kI8Tile + wq * 64;
  const int64_t c0 = kPairs<EPI> ? (int64_t)tp * (kI8Tile / 2) + wp * 32 : (int64_t)tp * kI8Tile + wp * 32 * PB;
  u32x4_t dh[QB][2];
  load_dh<EPI>(a, dh, r0, c0, lane);
  emit<T, EPI, PB, QB>(a, acc, dh, sc + wp * 64, sc + kI8Tile + wq * 64, r0, c0, lane, lds + wave * kOwnBytes, [] {});
}

// The tiles that were split: the sums of their parts, in order, and what the
// tile kernel does with sums.  A thread has four output columns of a row, and four parts on their way at a time.
template <class T, int EPI>
__global__ void __launch_bounds__(256)
k_i8_finish(TileArgs a, TilePlan pl) {
  using Sum = typename Mma<T>::Sum;
  constexpr int kCols = kPairs<EPI> ? 64 : 128, kChunks = kCols / 4, kRows = 256 / kChunks, kOuts = EPI == EPI_GATED_GRAD ? 2 : 1;
  constexpr int kHalves = kPairs<EPI> ? 2 : 1, kPart = kI8Tile * kI8Tile;
  constexpr int kBlocks = kI8Tile / kRows;         // of a tile
  const int split = blockIdx.x / kBlocks, r = (blockIdx.x % kBlocks) * kRows + threadIdx.x / kChunks;
  const int c = threadIdx.x % kChunks;
  int tp, tq;
  tile_at(pl.full + split, pl.tiles_p, pl.tiles_q, tp, tq);
  const int64_t row = (int64_t)tq * kI8Tile + r, col = (int64_t)tp * kCols + 4 * c;
  if (row >= a.rows || col >= a.cols) return;
  // place in the tile: pairs hold gate and up columns in blocks of 32
  const int p = kPairs<EPI> ? (c >> 3) * 64 + (c & 7) * 4 : 4 * c;
  const Sum* in = reinterpret_cast<const Sum*>(pl.part) + (int64_t)split * pl.cut * kPart + r * kI8Tile + p;
  Sum s[kHalves][4] = {};
  auto add = [&](const u32x4_t (&v)[kHalves]) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[h][e] += __builtin_bit_cast(Sum, (uint32_t)v[h][e]);
  };
  int i = 0;
  for (; i + 4 <= pl.cut; i += 4, in += 4 * kPart) {
    u32x4_t v[4][kHalves];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) v[u][h] = ld16(in + u * kPart + 32 * h);
#pragma unroll
    for (int u = 0; u < 4; ++u) add(v[u]);
  }
  for (; i < pl.cut; ++i, in += kPart) {
    u32x4_t v[kHalves];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) v[h] = ld16(in + 32 * h);
    add(v);
  }
  const float sq = std::is_same<T, int8_t>::value ? a.qs[row] : 1.0f;
  float f[kOuts][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t n = min(col + e, a.cols - 1);
    if constexpr (EPI == EPI_ROUND) {
      f[0][e] = s[0][e];
    } else if constexpr (EPI == EPI_SCALE) {
      f[0][e] = (float)s[0][e] * sq * a.ps[n];
    } else {
      const float g = (float)s[0][e] * sq * a.ps[n], u = (float)s[1][e] * sq * a.ps[a.cols + n];
      if constexpr (EPI == EPI_GATED) f[0][e] = gated(g, u);
      else gated_grad(g, u, bf16_to_f32(a.dh[row * a.cols + n]), f[0][e], f[1][e]);
    }
  }
#pragma unroll
  for (int k = 0; k < kOuts; ++k) {
    uint16_t* y = a.out + row * kOuts * a.cols + k * a.cols + col;
    const u32x2_t v = {pack_bf16(f[k][0], f[k][1]), pack_bf16(f[k][2], f[k][3])};
    if (col + 3 < a.cols) {
      *reinterpret_cast<u32x2_a2_t*>(y) = v;
    } else {
      for (int e = 0; col + e < a.cols; ++e) y[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
  }
}

template <class T, int PM, bool QS, int EPI, int ST>
hipError_t run(const TileArgs& a, const TilePlan& pl, unsigned blocks, hipStream_t st) {
  constexpr int kLds = kTileLds<PM == P_CODES, ST>;
  auto kern = &k_i8_tile<T, PM, QS, EPI, ST>;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(kern, dim3(blocks), dim3(ST == 4 ? 320 : 256), kLds, st, a, pl);
  return hipGetLastError();
}

template <class T, int PM, bool QS, int EPI>
hipError_t go(const TileArgs& a, const TilePlan& pl, hipStream_t st) {
  const int64_t split = (int64_t)pl.tiles_p * pl.tiles_q - pl.full;
  const int64_t blocks = 8 * (((int64_t)pl.full + 7) / 8 + (split * pl.cut + 7) / 8);
  const hipError_t e = pl.two ? run<T, PM, QS, EPI, 2>(a, pl, (unsigned)blocks, st) : run<T, PM, QS, EPI, 4>(a, pl, (unsigned)blocks, st);
  if (e != hipSuccess) return e;
  if (split) {
    const int per = kPairs<EPI> ? 8 : 16;          // blocks of a tile: 16 rows, 8 rows
    hipLaunchKernelGGL((&k_i8_finish<T, EPI>), dim3((unsigned)(split * per)), dim3(256), 0, st, a, pl);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_tile(const TileArgs& a, const TilePlan& pl, int kind, hipStream_t st) {
  switch (kind) {
    case I8_FORWARD: return go<int8_t, P_ROWS, false, EPI_SCALE>(a, pl, st);
    case I8_GATED: return go<int8_t, P_ROWS, false, EPI_GATED>(a, pl, st);
    case I8_GATED_GRAD: return go<int8_t, P_ROWS, false, EPI_GATED_GRAD>(a, pl, st);
    case I8_DX: return pl.codes ? go<uint16_t, P_CODES, false, EPI_ROUND>(a, pl, st) : go<uint16_t, P_BF16, false, EPI_ROUND>(a, pl, st);
    default: return pl.codes ? go<uint16_t, P_CODES, true, EPI_ROUND>(a, pl, st) : go<uint16_t, P_BF16, true, EPI_ROUND>(a, pl, st);
  }
}

}  // namespace hm
