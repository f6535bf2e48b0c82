// Pieces that the tile kernels of the 8-bit integer layers share: operand
// copies into LDS, operand reads, the order of tiles and the epilogues.
//
// LDS holds an operand in halves of 128 rows (of the output side) x 128 bytes
// of the contraction, 16 KiB:
//   contraction contiguous: row r at 128 r, its 16-byte chunk c at place
//     c ^ ((r >> 1) & 7): the 16-byte operand reads of 16 neighbouring rows then
//     meet every bank once;
//   contraction as rows (bf16, 64 rows c of 128 values): row c at 256 c, chunk x
//     at place x ^ 4 (c & 3): a transposing read takes 64 bytes of four
//     neighbouring rows, which so lie in different banks.
// The copies write LDS in lane order; the places come from which chunk a lane
// fetches, and every copy moves whole lines.
#pragma once
#include <hip/hip_runtime.h>

#include "common.h"
#include "i8.h"

namespace hm {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

constexpr int kHalfBytes = 16384;

// 32 x 32 products: lane L supplies row L % 32 of each operand, bytes 16 (L / 32) .. + 15
// of 32; the result has column (second operand) L % 32 and rows 8 j + 4 (L / 32) + r in
// register 4 j + r.
template <class T> struct Mma;
template <> struct Mma<int8_t> {
  using Acc = i32x16_t;
  static __device__ __forceinline__ Acc run(u32x4_t a, u32x4_t b, Acc c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
  }
};
template <> struct Mma<uint16_t> {   // bf16 patterns
  using Acc = f32x16_t;
  static __device__ __forceinline__ Acc run(u32x4_t a, u32x4_t b, Acc c) { return mfma32_bf16(a, b, c); }
};

// Tile of this block: the eight XCDs (block b runs on b % 8) get consecutive
// ranges of an order that goes through four tile rows together, so that the
// blocks of an L2 share operands.  False: no tile.
__device__ __forceinline__ bool tile_of(int tiles_p, int tiles_q, int& tp, int& tq) {
  const uint32_t total = (uint32_t)tiles_p * (uint32_t)tiles_q, x = blockIdx.x & 7;    // under 2^24
  const uint32_t t = x * total / 8 + (blockIdx.x >> 3);
  if (t >= (x + 1) * total / 8) return false;
  const uint32_t group = t / (4u * tiles_p), in = t - group * 4u * tiles_p;
  const uint32_t rows = min(4u, (uint32_t)tiles_q - 4u * group), c = in / rows;
  tq = (int)(4u * group + in - c * rows);
  tp = (int)c;
  return true;
}

// Gated products pair the gate and up rows in blocks of 32: row r of a tile is
// gate row (EPI_GATED*) 32 (r / 64) + r % 32 of the tile's for even r / 32, the up
// row of the same number for odd.  A tile of `size` rows covers size / 2 columns of h.
template <int EPI> constexpr bool kPairs = EPI == EPI_GATED || EPI == EPI_GATED_GRAD;
template <int EPI> __host__ __device__ inline int64_t p_tiles(int64_t cols, int size) {
  const int per = kPairs<EPI> ? size / 2 : size;
  return (cols + per - 1) / per;
}
// Row of the scales (clamped to the last) that row r of column tile tp has.
template <int EPI> __device__ __forceinline__ int64_t p_row(const TileArgs& a, int tp, int size, int r) {
  if (!kPairs<EPI>) return min((int64_t)tp * size + r, a.cols - 1);
  const int64_t c = min((int64_t)tp * (size / 2) + (r >> 6) * 32 + (r & 31), a.cols - 1);
  return ((r >> 5) & 1) ? a.cols + c : c;
}

// Copies of one operand.  ROWS: the contraction runs along the array's rows
// (else the array's rows are contracted).  A half takes four copies a wave.
template <bool ROWS, bool PAIRS> struct Side {
  const uint8_t* base;       // of this tile (PAIRS: of the wave's gate or up rows), at the next step
  int64_t left;              // bytes of the array from there
  uint32_t vo[2];            // lane offsets of copies i = 0, 1 of half 0
  uint32_t ld;
  uint32_t tail;             // all ones where the lane's chunk lies behind the contraction in the last step
  uint32_t cut;              // the tail of the current step
  rsrc_t r;

  __device__ __forceinline__ void init(const uint8_t* arr, int64_t ld_, int64_t bytes, int64_t rows, int tile, int size,
                                       int lane, int wave, int64_t kbytes) {
    ld = (uint32_t)ld_;
    int64_t at;
    tail = 0;
    if (ROWS) {
      // wave w copies rows 16 w .. + 15 of the 64 contracted, four at a time
      at = (int64_t)tile * size * 2;
      vo[0] = (uint32_t)(wave * 16 + (lane >> 4)) * ld + 16 * ((lane & 15) ^ (4 * ((lane >> 4) & 3)));
      vo[1] = vo[0] + 4 * ld;
    } else {
      // wave w copies rows 32 w .. + 31 of a half, eight at a time
      const int first = PAIRS ? (wave >> 1) * 32 : wave * 32;
      if (PAIRS && (wave & 1)) arr += bytes;          // the up rows, behind the gate rows
      at = (int64_t)tile * (PAIRS ? size / 2 : size) * ld_;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int chunk = (lane & 7) ^ ((lane >> 4) | (4 * i));
        vo[i] = (uint32_t)(first + 8 * i + (lane >> 3)) * ld + 16 * chunk;
      }
      // whether the chunk's bytes of the last step end behind the contraction (copies i = 0 and 1 differ in chunk)
      const int in = (int)(kbytes & 127);
      if (in) {
        tail = ((16 * ((lane & 7) ^ (lane >> 4))) >= in ? 1u : 0u) | ((16 * ((lane & 7) ^ ((lane >> 4) | 4))) >= in ? 2u : 0u);
      }
    }
    base = arr + at;
    left = bytes - at;
    cut = 0;
    (void)rows;
  }
  // The array as step s sees it (steps follow each other from 0); behind the last step everything reads as zero.
  __device__ __forceinline__ void step(int s, int steps) {
    r = make_rsrc(base, s < steps && left > 0 ? (uint64_t)left : 0);
    cut = s == steps - 1 ? tail : 0;
    const int64_t by = ROWS ? 64 * (int64_t)ld : 128;
    base += by;
    left -= by;
  }
  // Copy i (0..3) of half h to the half's place in LDS.
  __device__ __forceinline__ void copy(int h, int i, uint8_t* half, int wave) {
    if (ROWS) {
      b2lds16(r, vo[i & 1] + (uint32_t)(i & 2) * 4 * ld + (uint32_t)h * 256, 0u, half + (wave * 16 + i * 4) * 256);
    } else {
      const uint32_t over = (cut >> (i & 1)) & 1u ? 0xFFFFFFFFu : 0u;
      b2lds16(r, (vo[i & 1] + ((uint32_t)(i & 2) * 8 + (uint32_t)h * (PAIRS ? 64 : 128)) * ld) | over, 0u,
              half + (wave * 32 + i * 8) * 128);
    }
  }
};

// Operand reads: block b (32 rows) of the wave's 64 rows of a half (w = 0, 1), part ks of the step's four.
template <bool ROWS> struct Frags {
  uint32_t at[4];
  __device__ __forceinline__ void init(int lane, int w) {
    if (ROWS) {
      // group of 16 lanes: columns 16 (g & 1) .., contraction 8 (g >> 1) ..; lane l of it fetches row l / 4, four columns
      const int g = lane >> 4, l = lane & 15;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int chunk = (w * 8 + b * 4 + 2 * (g & 1) + ((l & 3) >> 1)) ^ (4 * (l >> 2));
        at[b] = (uint32_t)((8 * (g >> 1) + (l >> 2)) * 256 + chunk * 16 + (l & 1) * 8);
      }
      at[2] = at[3] = 0;
    } else {
      const int l32 = lane & 31, hi = lane >> 5;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        at[ks] = (uint32_t)((w * 64 + l32) * 128 + 16 * ((2 * ks + hi) ^ ((l32 >> 1) & 7)));
    }
  }
  __device__ __forceinline__ u32x4_t read(const uint8_t* half, int b, int ks) const {
    if (ROWS) {
      const uint8_t* p = half + at[b] + ks * 16 * 256;
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p);
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 4 * 256));
      const u32x2_t x = __builtin_bit_cast(u32x2_t, lo), y = __builtin_bit_cast(u32x2_t, hi);
      return (u32x4_t){x[0], x[1], y[0], y[1]};
    }
    return ld16(half + at[ks] + b * 32 * 128);
  }
};

// Gate, up and the gradient of h to those of both, with sig = 1 / (1 + e^-g)
// from e = e^-|g| <= 1, so that neither sig nor 1 - sig overflows or cancels.
// Beyond |g| = 64, where e would leave the normal range, e 2^64 is held and the
// results of negative gates are scaled back last.  The fast exponential and
// the hardware reciprocal (a few 2^-23 together) stay far below the bf16
// rounding of the results.
__device__ __forceinline__ void gated_grad(float g, float u, float dh, float& dg, float& du) {
  const bool far = fabsf(g) > 64.0f, pos = g >= 0.0f;
  const float back = far ? 5.421010862427522e-20f : 1.0f;
  const float e = __expf((far ? 44.3614195558365f : 0.0f) - fabsf(g));
  const float s = __builtin_amdgcn_rcpf(1.0f + e * back), es = e * s;
  const float sig = pos ? s : es, last = pos ? 1.0f : back;
  const float rest = pos ? es * back : s;                              // 1 - sig
  du = dh * (g * sig) * last;
  dg = dh * u * (sig * __builtin_fmaf(g, rest, 1.0f)) * last;
}

// The tile's results through LDS (which the copies no longer use) to global memory in whole rows.
// H halves a side: wave (wp, wq) holds rows 128 h + 64 w + 32 b + ... of each side.
template <class T, int EPI, int H> struct Epilogue {
  using Acc = typename Mma<T>::Acc;
  static constexpr int kSize = 128 * H;                         // rows of the tile, and columns (pairs: of gate and up)
  static constexpr int kCols = kPairs<EPI> ? kSize / 2 : kSize;  // columns of each output
  static constexpr int kRowBytes = 2 * kCols, kChunks = kRowBytes / 16;
  const TileArgs& a;
  uint8_t* lds;
  const float *ps, *qs;                                         // the tile's scales
  int tp, tq, lane, wave, wp, wq, tid;

  // 16-byte chunk c of row r
  __device__ __forceinline__ int place(int r, int c) const { return r * kRowBytes + 16 * (c ^ (r & (kChunks - 1))); }

  // dh into LDS (EPI_GATED_GRAD)
  __device__ __forceinline__ void before() {
    if (EPI != EPI_GATED_GRAD) return;
    const int64_t c0 = (int64_t)tp * kCols, r0 = (int64_t)tq * kSize;
    for (int i = tid; i < kSize * kChunks; i += 256) {
      const int r = i / kChunks, c = i % kChunks;
      const int64_t row = r0 + r, col = c0 + 8 * c;
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (row < a.rows) {
        const uint16_t* src = a.dh + row * a.cols;
        if ((a.cols & 7) == 0 && col + 7 < a.cols) {
          v = ld16(src + col);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (col + e < a.cols) v[e >> 1] |= (uint32_t)src[col + e] << (16 * (e & 1));
        }
      }
      st16(lds + place(r, c), v);
    }
    __syncthreads();
  }

  // The wave's blocks of P half ph and Q half qh.
  __device__ __forceinline__ void put(int ph, int qh, const Acc (&acc)[2][2]) {
    const int l32 = lane & 31, hi = lane >> 5;
#pragma unroll
    for (int qb = 0; qb < 2; ++qb) {
      const int r = qh * 128 + wq * 64 + qb * 32 + l32;
      if (kPairs<EPI>) {
        const int c0 = (ph * 2 + wp) * 32;
        const float sq = qs[r];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = 8 * j + 4 * hi;
          const f32x4_t sg = *reinterpret_cast<const f32x4_t*>(ps + 2 * c0 + n);
          const f32x4_t su = *reinterpret_cast<const f32x4_t*>(ps + 2 * c0 + 32 + n);
          float g[4], u[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            g[e] = (float)acc[0][qb][4 * j + e] * sq * sg[e];
            u[e] = (float)acc[1][qb][4 * j + e] * sq * su[e];
          }
          uint8_t* at = lds + place(r, (c0 + n) >> 3) + 8 * hi;
          if (EPI == EPI_GATED) {
            float h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = silu_f(g[e]) * u[e];
            *reinterpret_cast<u32x2_t*>(at) = (u32x2_t){pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3])};
          } else {
            const u32x2_t d = *reinterpret_cast<const u32x2_t*>(at);
            float dg[4], du[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              gated_grad(g[e], u[e], (e & 1) ? hi_bf16(d[e >> 1]) : lo_bf16(d[e >> 1]), dg[e], du[e]);
            *reinterpret_cast<u32x2_t*>(at) = (u32x2_t){pack_bf16(dg[0], dg[1]), pack_bf16(dg[2], dg[3])};
            *reinterpret_cast<u32x2_t*>(at + kSize * kRowBytes) = (u32x2_t){pack_bf16(du[0], du[1]), pack_bf16(du[2], du[3])};
          }
        }
      } else {
#pragma unroll
        for (int pb = 0; pb < 2; ++pb) {
          const int c0 = ph * 128 + wp * 64 + pb * 32;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int n = 8 * j + 4 * hi;
            float y[4];
            if (EPI == EPI_SCALE) {
              const float sq = qs[r];
              const f32x4_t sp = *reinterpret_cast<const f32x4_t*>(ps + c0 + n);
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = (float)acc[pb][qb][4 * j + e] * sq * sp[e];
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = acc[pb][qb][4 * j + e];
            }
            *reinterpret_cast<u32x2_t*>(lds + place(r, (c0 + n) >> 3) + 8 * hi) =
                (u32x2_t){pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
          }
        }
      }
    }
  }

  __device__ __forceinline__ void store() {
    __syncthreads();
    const int64_t c0 = (int64_t)tp * kCols, r0 = (int64_t)tq * kSize;
    constexpr int kOuts = EPI == EPI_GATED_GRAD ? 2 : 1;
    const int64_t ld = kOuts * a.cols;
    for (int i = tid; i < kSize * kChunks; i += 256) {
      const int r = i / kChunks, c = i % kChunks;
      const int64_t row = r0 + r, col = c0 + 8 * c;
      if (row >= a.rows || col >= a.cols) continue;
#pragma unroll
      for (int o = 0; o < kOuts; ++o)
        store_row8(a.out + row * ld + o * a.cols, ld, a.cols, col, ld16(lds + place(r, c) + o * kSize * kRowBytes));
    }
  }
  // Eight values of a row at col (those under cols): one store where rows and halves are 16-byte aligned.
  static __device__ __forceinline__ void store_row8(uint16_t* y, int64_t ld, int64_t cols, int64_t col, u32x4_t v) {
    if ((ld & 7) == 0 && (cols & 7) == 0 && col + 7 < cols) {
      st16(y + col, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e < cols) y[col + e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
  }
};

}  // namespace hm
