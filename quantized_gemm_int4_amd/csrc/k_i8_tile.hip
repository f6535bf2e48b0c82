// Products of 8-bit integer layers and of their gradients, 128 x 128 output
// tiles: O[q][p] = sum_c Q[q][c] P[p][c] on 32x32 MFMAs, int8 codes with exact
// integer sums (32x32x32) or bf16 with fp32 sums (32x32x16).
//
// A block of four waves, each with 64 x 64 of the tile.  The MFMA's rows are the
// output's columns p, so that a lane holds four neighbouring columns of one
// output row.  Operands come through LDS in steps of 128 bytes of the
// contraction by 16-byte direct buffer-to-LDS copies; reads past an array give
// zeros, so no size has to be padded.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "common.h"
#include "i8.h"
#include "i8_tile.h"

namespace hm {

namespace {

constexpr int kStage = 2 * kHalfBytes;             // P and Q of one step
constexpr int kTileLds = 2 * kStage + 1024;        // two stages, 128 + 128 scales

template <class T, bool PS, bool QS, int EPI>
__global__ void __launch_bounds__(256, 2)
k_i8_tile(TileArgs a, int tiles_p, int tiles_q) {
  using Acc = typename Mma<T>::Acc;
  extern __shared__ __align__(1024) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wave & 1, wq = wave >> 1;
  int tp, tq;
  if (!tile_of(tiles_p, tiles_q, tp, tq)) return;
  float* sc = reinterpret_cast<float*>(lds + 2 * kStage);
  if (std::is_same<T, int8_t>::value) {
    if (tid < kI8Tile) sc[tid] = a.ps[p_row<EPI>(a, tp, kI8Tile, tid)];
    else sc[tid] = a.qs[min((int64_t)tq * kI8Tile + tid - kI8Tile, a.rows - 1)];
  }
  Side<PS, EPI == EPI_GATED || EPI == EPI_GATED_GRAD> P;
  Side<QS, false> Q;
  P.init(a.p, a.p_ld, a.p_bytes, a.cols, tp, kI8Tile, lane, wave, a.kbytes);
  Q.init(a.q, a.q_ld, a.q_bytes, a.rows, tq, kI8Tile, lane, wave, a.kbytes);
  const int steps = (int)((a.kbytes + 127) / 128);

  Acc acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  auto copy = [&](int s) __attribute__((always_inline)) {
    uint8_t* st = lds + (s & 1) * kStage;
    P.step(s, steps);
    Q.step(s, steps);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      P.copy(0, i, st, wave);
      Q.copy(0, i, st + kHalfBytes, wave);
    }
  };
  Frags<PS> fp;
  Frags<QS> fq;
  fp.init(lane, wp);
  fq.init(lane, wq);
  copy(0);
  for (int s = 0; s < steps; ++s) {
    // this step's copies have landed and every wave has read the stage that the next ones go to
    __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (s + 1 < steps) copy(s + 1);
    const uint8_t* st = lds + (s & 1) * kStage;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      u32x4_t vp[2], vq[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        vp[b] = fp.read(st, b, ks);
        vq[b] = fq.read(st + kHalfBytes, b, ks);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = Mma<T>::run(vp[i], vq[j], acc[i][j]);
    }
  }
  __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  Epilogue<T, EPI, 1> ep{a, lds, sc, sc + kI8Tile, tp, tq, lane, wave, wp, wq, tid};
  ep.before();
  ep.put(0, 0, acc);
  ep.store();
}

template <class T, bool PS, bool QS, int EPI>
hipError_t go(const TileArgs& a, hipStream_t st) {
  auto kern = &k_i8_tile<T, PS, QS, EPI>;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, kTileLds);
  if (attr != hipSuccess) return attr;
  const int64_t tp = p_tiles<EPI>(a.cols, kI8Tile), tq = (a.rows + kI8Tile - 1) / kI8Tile;
  hipLaunchKernelGGL(kern, dim3((unsigned)(8 * ((tp * tq + 7) / 8))), dim3(256), kTileLds, st, a, (int)tp, (int)tq);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_tile(const TileArgs& a, int kind, hipStream_t st) {
  switch (kind) {
    case I8_FORWARD: return go<int8_t, false, false, EPI_SCALE>(a, st);
    case I8_GATED: return go<int8_t, false, false, EPI_GATED>(a, st);
    case I8_GATED_GRAD: return go<int8_t, false, false, EPI_GATED_GRAD>(a, st);
    case I8_DX: return go<uint16_t, true, false, EPI_ROUND>(a, st);
    default: return go<uint16_t, true, true, EPI_ROUND>(a, st);
  }
}

}  // namespace hm
