// The products of k_i8_tile.hip on 256 x 256 output tiles, for calls with
// tiles enough to fill the card: the matrix cores are busy in 61 % of its cycles, and power sets the clock (int8
// product m = 8192, n = 14336, k = 4096, calls in a row, two cards: 399 and 407 us with Gaussian codes, 2.4 Pop/s at about 1.9 GHz, 296 with
// zeros; gated block m = 4096 409 and 419, its gradient 459, with an epilogue of four bf16 results a pair; bf16 gradients m = 4096, same n and
// k, one call at a time: 366 and 377 us dx, 396 and 410 dw, 1.27 to 1.31 and 1.17 to 1.22 PFLOP/s).
//
// Four waves, one per SIMD, each with 128 x 128 of the tile (256 accumulators a
// lane): every 16-byte operand read from LDS feeds two (halves: four) MFMAs.  A read of 1 KiB takes
// LDS four cycles (its counter), so a step of 128 bytes has 512 cycles of reads for 2048 of MFMA, and 64 KiB of
// copies into LDS.  (64 x 64 a wave, as in the 128 x 128 kernel: 256 for 512, and 32 KiB.)
//
// A step is cut into four phases, one for each pair of P and Q halves, 16 MFMAs of 32
// cycles each.  Every phase reads the operands of the next one between its
// MFMAs and issues the copies of a quarter of the step after the next:
//   phase   MFMAs      operand reads       copies
//     0     P0 Q0      Q1 of this step     P0 of step s + 2
//     1     P0 Q1      P1 of this step     Q0 of step s + 2
//     2     P1 Q1      P0 of step s + 1    Q1 of step s + 2
//     3     P1 Q0      Q0 of step s + 1    P1 of step s + 2
// LDS has two stages; the halves of step s + 2 go where those of step s were:
// P0 and Q0 have been read by phase 0 of step s (in phases 2 and 3 of step s - 1),
// Q1 and P1 by phase 2, and a barrier before phases 0 and 2 says so for all
// waves.  The same barriers, with all but the newest 16 copies waited for, say
// that the halves read until the next one have landed: four phases, 2048 cycles,
// after the last of them was issued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "common.h"
#include "i8.h"
#include "i8_tile.h"

namespace hm {

namespace {

constexpr int kBigStage = 4 * kHalfBytes;              // P0, P1, Q0, Q1
constexpr int kBigOwn = 2 * kBigStage + 2048;          // two stages, 256 + 256 scales; then 4 KiB a wave for its results
constexpr int kBigLds = kBigOwn + 4 * kOwnBytes;

template <class T, bool PS, bool QS, int EPI>
__global__ void __launch_bounds__(256, 1)
k_i8_big(TileArgs a, int tiles_p, int tiles_q) {
  using Acc = typename Mma<T>::Acc;
  constexpr bool I8 = std::is_same<T, int8_t>::value;
  extern __shared__ __align__(1024) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wave & 1, wq = wave >> 1;
  float* sc = reinterpret_cast<float*>(lds + 2 * kBigStage);
  const int steps = (int)((a.kbytes + 127) / 128);
  int tp, tq, turn = 0;
  if (!tile_of(tiles_p * tiles_q, gridDim.x, 0, tiles_p, tiles_q, tp, tq)) return;
  Side<PS, kPairs<EPI>> P;
  Side<QS, false> Q;
  Frags<PS> fp;
  Frags<QS> fq;
  fp.init(lds, lane, wp);
  fq.init(lds, lane, wq);

  P.init(a.p, a.p_ld, a.p_bytes, kI8Big, lane, wave, a.kbytes);
  Q.init(a.q, a.q_ld, a.q_bytes, kI8Big, lane, wave, a.kbytes);
  P.tile(tp);
  Q.tile(tq);
  // steps 0 and 1 of the first tile, in the order of the phases
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint8_t* st = lds + s * kBigStage;
    P.step(s, steps, steps);
    Q.step(s, steps, steps);
#pragma unroll
    for (int i = 0; i < 4; ++i) P.copy(0, i, st, wave);
#pragma unroll
    for (int i = 0; i < 4; ++i) Q.copy(0, i, st + 2 * kHalfBytes, wave);
#pragma unroll
    for (int i = 0; i < 4; ++i) Q.copy(1, i, st + 3 * kHalfBytes, wave);
#pragma unroll
    for (int i = 0; i < 4; ++i) P.copy(1, i, st + kHalfBytes, wave);
  }
  u32x4_t p0[2][4], p1[2][4], qa[2][4], qb[2][4];
  Acc acc[2][2][2][2];                                 // P half, Q half, blocks of each

  // 16 MFMAs of one pair of halves; after every second one an operand read
  // (in the order the next phase uses them), after every fourth a copy
  auto phase = [&](Acc (&c)[2][2], const u32x4_t (&vp)[2][4], const u32x4_t (&vq)[2][4], auto&& read, auto&& copy)
                   __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int ks = i >> 2, x = (i >> 1) & 1, y = i & 1;
      c[x][y] = Mma<T>::run(vp[x][ks], vq[y][ks], c[x][y]);
      if (i & 1) {
        read((i >> 1) & 1, i >> 2);
        if ((i & 3) == 3) copy(i >> 2);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  // all waves have read what they asked for, and all but the newest 16 copies have landed
  auto sync = [&](bool landed) __attribute__((always_inline)) {
    if (landed) __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else __asm__ volatile("s_waitcnt vmcnt(16) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  // one step; q0: this step's Q0, whose registers take nothing new before the
  // next step's Q1, q1: takes this step's Q1, then the next step's Q0
  // The first one and a half steps of a tile find their copies landed and wait for
  // none: the last tile's stores may still be on their way.  n: the step that is copied
  // during step s, of this tile or the next.
  auto step = [&](int s, int n, u32x4_t (&q0)[2][4], u32x4_t (&q1)[2][4], auto parity) __attribute__((always_inline)) {
    uint8_t* st = lds + parity.value * kBigStage;
    const uint32_t here = in_sgpr(parity.value * kBigStage), there = in_sgpr((1 - parity.value) * kBigStage);
    const Frags<PS> hp = fp.moved(here), np = fp.moved(there);
    const Frags<QS> hq = fq.moved(here), nq = fq.moved(there);
    P.step(n, steps, steps);
    Q.step(n, steps, steps);
    sync(s == parity.value);
    phase(acc[0][0], p0, q0, [&](int b, int ks) { q1[b][ks] = hq.read(3 * kHalfBytes, b, ks); },
          [&](int i) { P.copy(0, i, st, wave); });
    phase(acc[0][1], p0, q1, [&](int b, int ks) { p1[b][ks] = hp.read(kHalfBytes, b, ks); },
          [&](int i) { Q.copy(0, i, st + 2 * kHalfBytes, wave); });
    sync(parity.value == 0 && s == 0);
    phase(acc[1][1], p1, q1, [&](int b, int ks) { p0[b][ks] = np.read(0, b, ks); },
          [&](int i) { Q.copy(1, i, st + 3 * kHalfBytes, wave); });
    phase(acc[1][0], p1, q0, [&](int b, int ks) { q1[b][ks] = nq.read(2 * kHalfBytes, b, ks); },
          [&](int i) { P.copy(1, i, st + kHalfBytes, wave); });
  };
  __asm__ volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p0[i >> 2][i & 3] = fp.read(0, i >> 2, i & 3);
    qa[i >> 2][i & 3] = fq.read(2 * kHalfBytes, i >> 2, i & 3);
  }
  // Two steps a round, of which the last may be past the end and all zeros (one
  // way out of the loop: a second one costs the compiler copies of the
  // accumulators).  The last round copies and reads the next tile's first steps.
  const int rounds = max(1, (steps + 1) >> 1);
  while (true) {
    float sp = 0.f, sq = 0.f;
    if (I8) {
      sp = a.ps[p_row<EPI>(a, tp, kI8Big, tid)];
      sq = a.qs[min((int64_t)tq * kI8Big + tid, a.rows - 1)];
    }
    int np = -1, nq = -1;
    const bool more = tile_of(tiles_p * tiles_q, gridDim.x, ++turn, tiles_p, tiles_q, np, nq);
    if (!more) np = nq = -1;
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i >> 3][(i >> 2) & 1][(i >> 1) & 1][i & 1][r] = 0;
    int s = 0;
    do {
      int n = s + 2;
      if (n == 2 * rounds) {
        P.tile(np);
        Q.tile(nq);
        n = 0;
      }
      step(s, n, qa, qb, std::integral_constant<int, 0>());
      step(s + 1, n + 1, qb, qa, std::integral_constant<int, 1>());
      s += 2;
    } while (s < 2 * rounds);
    // the sums leave the loop where they are (else the compiler may move some out of the way in every round)
#pragma unroll
    for (int i = 0; i < 16; ++i) __asm__ volatile("" : "+a"(acc[i >> 3][(i >> 2) & 1][(i >> 1) & 1][i & 1]));
    if (I8) {
      sc[tid] = sp;
      sc[256 + tid] = sq;
      __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
    const int64_t r0 = (int64_t)tq * kI8Big + wq * 64;
    const int64_t c0 = kPairs<EPI> ? (int64_t)tp * (kI8Big / 2) + wp * 32 : (int64_t)tp * kI8Big + wp * 64;
    constexpr int kCols = kPairs<EPI> ? 64 : 128;      // output columns of a P half
    const int ln = (int)in_vgpr((uint32_t)lane);       // (what is worked out again needs no registers in between)
    u32x4_t dh[4][2][2];
#pragma unroll
    for (int h = 0; h < 4; ++h) load_dh<EPI>(a, dh[h], r0 + (h & 1) * 128, c0 + (h >> 1) * kCols, ln);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      // the copies land before the first store: the waits for them wait for no store
      emit<T, EPI, 2, 2>(a, acc[h >> 1][h & 1], dh[h], sc + (h >> 1) * 128 + wp * 64, sc + 256 + (h & 1) * 128 + wq * 64,
                   r0 + (h & 1) * 128, c0 + (h >> 1) * kCols, ln, lds + kBigOwn + wave * kOwnBytes, [&]() {
                     if (h == 0) __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
                   });
      __builtin_amdgcn_sched_barrier(0);
    }
    if (!more) break;
    tp = np;
    tq = nq;
  }
}

template <class T, bool PS, bool QS, int EPI>
hipError_t go(const TileArgs& a, hipStream_t st) {
  auto kern = &k_i8_big<T, PS, QS, EPI>;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, kBigLds);
  if (attr != hipSuccess) return attr;
  const int64_t tp = p_tiles<EPI>(a.cols, kI8Big), tq = (a.rows + kI8Big - 1) / kI8Big;
  // one block a compute unit, each through several tiles where there are more
  hipLaunchKernelGGL(kern, dim3((unsigned)std::min<int64_t>(256, 8 * ((tp * tq + 7) / 8))), dim3(256), kBigLds, st, a, (int)tp, (int)tq);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_big(const TileArgs& a, int kind, hipStream_t st) {
  switch (kind) {
    case I8_FORWARD: return go<int8_t, false, false, EPI_SCALE>(a, st);
    case I8_GATED: return go<int8_t, false, false, EPI_GATED>(a, st);
    case I8_GATED_GRAD: return go<int8_t, false, false, EPI_GATED_GRAD>(a, st);
    case I8_DX: return go<uint16_t, true, false, EPI_ROUND>(a, st);
    default: return go<uint16_t, true, true, EPI_ROUND>(a, st);
  }
}

}  // namespace hm
