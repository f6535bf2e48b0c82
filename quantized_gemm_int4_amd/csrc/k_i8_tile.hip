// Products of 8-bit integer layers and of their gradients, 128 x 128 output
// tiles: O[q][p] = sum_c Q[q][c] P[p][c] on 32x32 MFMAs, int8 codes with exact
// integer sums (32x32x32) or bf16 with fp32 sums (32x32x16).  For calls with too
// few 256 x 256 tiles to fill the card: bound by the latency of their copies.
//
// A block of four waves, one a SIMD, each with 64 x 64 of the tile.  The MFMA's
// rows are the output's columns p, so that a lane holds four neighbouring
// columns of one output row.  Operands come through LDS in steps of 128 bytes
// of the contraction by 16-byte direct buffer-to-LDS copies; reads past an
// array give zeros, so no size has to be padded.  Gradients read their int8
// operand (weights for dx, rows of x for dw) as it is and turn it into bf16 between
// the MFMAs: the copies are what bounds these tiles (MFMAs take 0.21 us of a step's 0.77), and the 256 x 256
// tiles' bf16 copy of the operand would cost more than the conversion.  During step s its operands are
// in registers, those of step s + 1 are read from LDS between the MFMAs, and four
// stages hold steps s + 1 .. s + 4, so that a copy has three steps to land.
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

constexpr int kStages = 4;
// P8: P is int8 codes whose rows are contracted (gradients); then a stage also has a slot of 64 scales for each wave
template <bool P8> constexpr int kP = P8 ? Codes::kBytes : kHalfBytes;
template <bool P8> constexpr int kStage = kP<P8> + kHalfBytes;             // P and Q of one step
template <bool P8> constexpr int kScales = kStages * kStage<P8>;           // the slots, or the scales of 128 + 128 results
template <bool P8> constexpr int kTileLds = kScales<P8> + (P8 ? kStages * 1024 : 1024);

template <class T, bool P8, bool QS, int EPI>
__global__ void __launch_bounds__(256, 1)
k_i8_tile(TileArgs a, TilePlan pl) {
  using Acc = typename Mma<T>::Acc;
  extern __shared__ __align__(1024) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wave & 1, wq = wave >> 1;
  const int all = (int)((a.kbytes + 127) / 128);
  const uint32_t whole = 8 * ((uint32_t)(pl.full + 7) / 8);
  int tp, tq, first = 0, last = all, item = -1;
  if (blockIdx.x < whole) {
    if (!tile_of(pl.full, whole, 0, pl.tiles_p, pl.tiles_q, tp, tq)) return;
  } else {
    item = blockIdx.x - whole;
    tile_at(pl.full + item / pl.cut, pl.tiles_p, pl.tiles_q, tp, tq);
    first = (item % pl.cut) * pl.per;
    last = min(all, first + pl.per);
  }
  const int steps = last - first;
  float* sc = reinterpret_cast<float*>(lds + kScales<P8>);
  if (std::is_same<T, int8_t>::value) {
    if (tid < kI8Tile) sc[tid] = a.ps[p_row<EPI>(a, tp, kI8Tile, tid)];
    else sc[tid] = a.qs[min((int64_t)tq * kI8Tile + tid - kI8Tile, a.rows - 1)];
  }
  Side<QS, false> Q;
  Q.init(a.q, a.q_ld, a.q_bytes, kI8Tile, lane, wave, a.kbytes);
  Q.tile(tq, first);
  Frags<QS> fq;
  fq.init(lds + kP<P8>, lane, wq);
  std::conditional_t<P8, Codes, Side<false, kPairs<EPI>>> P;
  Frags<false> fp;
  uint8_t* const slot = lds + kScales<P8> + wave * 256;
  if constexpr (P8) {
    P.init(a.p, a.p_ld, a.p_bytes, a.ps, a.terms, tp, first, lane, wave, lds, slot);
  } else {
    P.init(a.p, a.p_ld, a.p_bytes, kI8Tile, lane, wave, a.kbytes);
    P.tile(tp, first);
    fp.init(lds, lane, wp);
  }

  Acc acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
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
  for (int s = 0; s < kStages; ++s) {
    begin(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) copy(i, s);
  }
  // Operands of a step in registers (codes as they are, with their scales).
  struct Ops {
    std::conditional_t<P8, u32x2_t, u32x4_t> p[2][4];
    u32x4_t q[2][4];
    f32x4_t s[4][2];
  };
  // part i = 0..7 of a step's operands, from the stage `by` bytes on
  auto read = [&](Ops& o, int i, int stage) __attribute__((always_inline)) {
    const int b = i & 1, ks = i >> 1;
    if constexpr (P8) {
      o.p[b][ks] = P.read(stage * kStage<P8>, b, ks);
      o.s[ks][b] = P.scales(stage * 1024, ks, b);
    } else {
      o.p[b][ks] = fp.moved(stage * kStage<P8>).read(0, b, ks);
    }
    o.q[b][ks] = fq.moved(stage * kStage<P8>).read(0, b, ks);
  };
  Ops a0, a1;
  __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(3 * kCopies) : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) read(a0, i, 0);
  // one step on operands o, while those of the next are read and step s + 4 is copied
  int at = 0;                                      // stage of step s
  auto step = [&](int s, const Ops& o, Ops& next) __attribute__((always_inline)) {
    const int after = (at + 1) & (kStages - 1);
    begin(s + kStages);
    // step s + 1 has landed (two steps' copies are newer), and all waves hold step s in registers
    __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(2 * kCopies) : "memory");
    u32x4_t vp[2][2];                              // P operands of parts ks and ks + 1
    auto values = [&](int b, int ks) __attribute__((always_inline)) {
      if constexpr (P8) vp[ks & 1][b] = Codes::values(o.p[b][ks], o.s[ks][0], o.s[ks][1]);
      else vp[ks & 1][b] = o.p[b][ks];
    };
    values(0, 0);
    values(1, 0);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int ks = i >> 2, x = (i >> 1) & 1, y = i & 1;
      acc[x][y] = Mma<T>::run(vp[ks & 1][x], o.q[y][ks], acc[x][y]);
      if (i & 1) read(next, i >> 1, after);
      else copy(i >> 1, at);
      if ((i & 1) && ks < 3) values((i >> 1) & 1, ks + 1);
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
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u32x4_t v;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const typename Mma<T>::Sum one = acc[x][y][4 * j + e];
            v[e] = __builtin_bit_cast(uint32_t, one);
          }
          st16(out + (wq * 64 + y * 32 + (lane & 31)) * kI8Tile + wp * 64 + x * 32 + 8 * j + 4 * (lane >> 5), v);
        }
    return;
  }
  const int64_t r0 = (int64_t)tq * kI8Tile + wq * 64;
  const int64_t c0 = kPairs<EPI> ? (int64_t)tp * (kI8Tile / 2) + wp * 32 : (int64_t)tp * kI8Tile + wp * 64;
  emit<T, EPI>(a, acc, sc + wp * 64, sc + kI8Tile + wq * 64, r0, c0, lane, lds + wave * kOwnBytes, [] {});
}

// The tiles that were split: the sums of their parts, in order, and what the
// tile kernel does with sums.  A thread has eight output columns of a row.
template <class T, int EPI>
__global__ void __launch_bounds__(256)
k_i8_finish(TileArgs a, TilePlan pl) {
  using Sum = typename Mma<T>::Sum;
  constexpr int kCols = kPairs<EPI> ? 64 : 128, kChunks = kCols / 8, kRows = 256 / kChunks, kOuts = EPI == EPI_GATED_GRAD ? 2 : 1;
  constexpr int kBlocks = kI8Tile / kRows;         // of a tile
  const int split = blockIdx.x / kBlocks, r = (blockIdx.x % kBlocks) * kRows + threadIdx.x / kChunks;
  const int c = threadIdx.x % kChunks;
  int tp, tq;
  tile_at(pl.full + split, pl.tiles_p, pl.tiles_q, tp, tq);
  const int64_t row = (int64_t)tq * kI8Tile + r, col = (int64_t)tp * kCols + 8 * c;
  if (row >= a.rows || col >= a.cols) return;
  // place in the tile: pairs hold gate and up columns in blocks of 32
  const int p = kPairs<EPI> ? (c >> 2) * 64 + (c & 3) * 8 : 8 * c;
  const Sum* in = reinterpret_cast<const Sum*>(pl.part) + (int64_t)split * pl.cut * kI8Tile * kI8Tile + r * kI8Tile + p;
  Sum s[kPairs<EPI> ? 2 : 1][8] = {};
  for (int i = 0; i < pl.cut; ++i, in += kI8Tile * kI8Tile) {
#pragma unroll
    for (int h = 0; h < (kPairs<EPI> ? 2 : 1); ++h) {
      const u32x4_t lo = ld16(in + 32 * h), hi = ld16(in + 32 * h + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[h][e] += __builtin_bit_cast(Sum, (uint32_t)lo[e]);
        s[h][4 + e] += __builtin_bit_cast(Sum, (uint32_t)hi[e]);
      }
    }
  }
  const float sq = std::is_same<T, int8_t>::value ? a.qs[row] : 1.0f;
  float f[kOuts][8];
  u32x4_t d = {0u, 0u, 0u, 0u};
  if (EPI == EPI_GATED_GRAD) d = load8(a.dh + row * a.cols, a.cols, col);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t n = min(col + e, a.cols - 1);
    if constexpr (EPI == EPI_ROUND) {
      f[0][e] = s[0][e];
    } else if constexpr (EPI == EPI_SCALE) {
      f[0][e] = (float)s[0][e] * sq * a.ps[n];
    } else {
      const float g = (float)s[0][e] * sq * a.ps[n], u = (float)s[1][e] * sq * a.ps[a.cols + n];
      if constexpr (EPI == EPI_GATED) f[0][e] = silu_f(g) * u;
      else gated_grad(g, u, (e & 1) ? hi_bf16(d[e >> 1]) : lo_bf16(d[e >> 1]), f[0][e], f[1][e]);
    }
  }
#pragma unroll
  for (int k = 0; k < kOuts; ++k) {
    u32x4_t v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pack_bf16(f[k][2 * e], f[k][2 * e + 1]);
    store8(a.out + row * kOuts * a.cols + k * a.cols, a.cols, col, v);
  }
}

template <class T, bool P8, bool QS, int EPI>
hipError_t go(const TileArgs& a, const TilePlan& pl, hipStream_t st) {
  auto kern = &k_i8_tile<T, P8, QS, EPI>;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, kTileLds<P8>);
  if (attr != hipSuccess) return attr;
  const int64_t split = (int64_t)pl.tiles_p * pl.tiles_q - pl.full;
  const int64_t blocks = 8 * (((int64_t)pl.full + 7) / 8) + split * pl.cut;
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256), kTileLds<P8>, st, a, pl);
  if (split) {
    const int per = kPairs<EPI> ? 4 : 8;           // blocks of a tile: 32 rows, 16 rows
    hipLaunchKernelGGL((&k_i8_finish<T, EPI>), dim3((unsigned)(split * per)), dim3(256), 0, st, a, pl);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_tile(const TileArgs& a, const TilePlan& pl, int kind, hipStream_t st) {
  switch (kind) {
    case I8_FORWARD: return go<int8_t, false, false, EPI_SCALE>(a, pl, st);
    case I8_GATED: return go<int8_t, false, false, EPI_GATED>(a, pl, st);
    case I8_GATED_GRAD: return go<int8_t, false, false, EPI_GATED_GRAD>(a, pl, st);
    case I8_DX: return go<uint16_t, true, false, EPI_ROUND>(a, pl, st);
    default: return go<uint16_t, true, true, EPI_ROUND>(a, pl, st);
  }
}

}  // namespace hm
