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
//     neighbouring rows, which so lie in different banks;
//   the same of int8 codes (64 rows of 128 bytes, 8 KiB): row c at 128 c, chunk x at
//     place x ^ 2 ((c >> 1) & 3): 32 bytes of eight neighbouring rows.
// The copies write LDS in lane order; the places come from which chunk a lane
// fetches, and every copy moves whole lines.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

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
  using Sum = int32_t;
  static __device__ __forceinline__ Acc run(u32x4_t a, u32x4_t b, Acc c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
  }
};
template <> struct Mma<uint16_t> {   // bf16 patterns
  using Acc = f32x16_t;
  using Sum = float;
  static __device__ __forceinline__ Acc run(u32x4_t a, u32x4_t b, Acc c) { return mfma32_bf16(a, b, c); }
};

// Tile number t of an order that goes through four tile rows together, so that
// blocks that run together share operands.
__device__ __forceinline__ void tile_at(uint32_t t, int tiles_p, int tiles_q, int& tp, int& tq) {
  const uint32_t group = t / (4u * tiles_p), in = t - group * 4u * tiles_p;
  const uint32_t rows = min(4u, (uint32_t)tiles_q - 4u * group), c = in / rows;
  tq = (int)(4u * group + in - c * rows);
  tp = (int)c;
}
// A block's number among `total` (under 2^24) that are dealt out to `blocks` blocks (a
// multiple of 8) over several turns, so that the eight XCDs (block b runs on b % 8) get
// consecutive ranges, and with them operands of their own L2s.  total: none.
__device__ __forceinline__ uint32_t number_of(uint32_t total, uint32_t block, uint32_t blocks, uint32_t turn) {
  const uint32_t x = block & 7, t = x * total / 8 + (block >> 3) + turn * (blocks >> 3);
  return t < (x + 1) * total / 8 ? t : total;
}
__device__ __forceinline__ bool tile_of(uint32_t total, uint32_t blocks, uint32_t turn, int tiles_p, int tiles_q, int& tp, int& tq) {
  const uint32_t t = number_of(total, blockIdx.x, blocks, turn);
  if (t >= total) return false;
  tile_at(t, tiles_p, tiles_q, tp, tq);
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
  const uint8_t* arr;        // PAIRS: the wave's gate or up rows
  int64_t bytes, per_tile;   // of the array, from one tile to the next
  const uint8_t* base;       // of the tile, at the next step
  int64_t left;              // bytes of the array from there
  uint32_t vo[2];            // lane offsets of copies i = 0, 1 of half 0
  uint32_t ld, ldv;          // bytes between rows; the same, unknown to the compiler (it would hold every copy's offset in a register)
  uint32_t tail, cut;        // bit i: the lane's chunk of copies i, i + 2 lies behind the contraction in the last step; in this one
  rsrc_t r;

  __device__ __forceinline__ void init(const uint8_t* arr_, int64_t ld_, int64_t bytes_, int size, int lane, int wave, int64_t kbytes) {
    arr = arr_;
    bytes = bytes_;
    ld = (uint32_t)ld_;
    tail = 0;
    if (ROWS) {
      // wave w copies rows 16 w .. + 15 of the 64 contracted, four at a time
      per_tile = size * 2;
      vo[0] = (uint32_t)(wave * 16 + (lane >> 4)) * ld + 16 * ((lane & 15) ^ (4 * ((lane >> 4) & 3)));
      vo[1] = vo[0] + 4 * ld;
    } else {
      // wave w copies rows 32 w .. + 31 of a half, eight at a time
      const int first = PAIRS ? (wave >> 1) * 32 : wave * 32;
      if (PAIRS && (wave & 1)) arr += bytes;          // the up rows, behind the gate rows
      per_tile = (PAIRS ? size / 2 : size) * ld_;
      const int in = (int)(kbytes & 127);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int chunk = (lane & 7) ^ ((lane >> 4) | (4 * i));
        vo[i] = (uint32_t)(first + 8 * i + (lane >> 3)) * ld + 16 * chunk;
        if (in && 16 * chunk >= in) tail |= 1u << i;
      }
    }
    cut = 0;
  }
  // Goes to step s of a tile; none (t < 0): everything reads as zero.
  __device__ __forceinline__ void tile(int t, int s = 0) {
    const int64_t at = t * per_tile + s * (ROWS ? 64 * (int64_t)ld : 128);
    base = arr + (t < 0 ? 0 : at);
    left = t < 0 ? 0 : bytes - at;
  }
  // The array as step s of `all` sees it (steps follow each other); from step `last` on everything reads as zero.
  __device__ __forceinline__ void step(int s, int last, int all) {
    r = make_rsrc(base, s < last && left > 0 ? (uint64_t)left : 0);
    cut = s == all - 1 ? tail : 0;
    ldv = in_sgpr(ld);
    const int64_t by = ROWS ? 64 * (int64_t)ld : 128;
    base += by;
    left -= by;
  }
  // Copy i (0..3) of half h to the half's place in LDS.
  __device__ __forceinline__ void copy(int h, int i, uint8_t* half, int wave) {
    if (ROWS) {
      b2lds16(r, vo[i & 1] + (uint32_t)(i & 2) * 4 * ldv + (uint32_t)h * 256, 0u, half + (wave * 16 + i * 4) * 256);
    } else {
      const uint32_t over = (cut >> (i & 1)) & 1u ? 0xFFFFFFFFu : 0u;
      b2lds16(r, (vo[i & 1] + ((uint32_t)(i & 2) * 8 + (uint32_t)h * (PAIRS ? 64 : 128)) * ldv) | over, 0u,
              half + (wave * 32 + i * 8) * 128);
    }
  }
};

// A transposing read of 16 x 4 values by 16 lanes: lane l supplies the address of row l / 4, columns 4 (l % 4) .. + 3, and gets
// column l of the four rows.  The restrict gives the read alias information; without any the compiler waits for every
// copy into LDS that is in flight (the gradient of m = 4096, n = 14336, k = 4096: 2303 us).
__device__ __forceinline__ u32x2_t read_tr16(const lds_s16x4_t* __restrict__ p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(const_cast<lds_s16x4_t*>(p)));
}

// The same of 16 x 8 bytes: lane l supplies the address of row l / 2, bytes 8 (l % 2) .. + 7, and gets byte l of the eight rows.
typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2_t lds_i32x2_t;
__device__ __forceinline__ u32x2_t read_tr8(const lds_i32x2_t* __restrict__ p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr8_b64_v2i32(const_cast<lds_i32x2_t*>(p)));
}

// Touches 128-byte lines of later steps, so that the copies find them in their
// XCD's L2 (a line from further away takes longer than a copy has).  The `sharers`
// blocks that run on the same rows divide a step's lines: this one has lines share,
// share + sharers, ...  A touch is a 4-byte copy a line to a place in LDS that nothing reads.
struct Ahead {
  const uint8_t* base;       // of the tile, at the next step
  int64_t left, by;          // bytes of the array from there, from one step to the next
  uint32_t vo[2];
  bool two;                  // more than 64 lines

  // from: bytes to the tile's first line; per_row lines in each of the rows, `ld` bytes apart
  __device__ __forceinline__ void init(const uint8_t* arr, int64_t bytes, int64_t from, int64_t by_, int64_t ld, int lines,
                                       int per_row, int share, int sharers, int lane) {
    base = arr + from;
    left = bytes - from;
    by = by_;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = (lane + 64 * i) * sharers + share;
      vo[i] = j < lines ? (uint32_t)(j / per_row) * (uint32_t)ld + 128 * (j % per_row) : 0xFFFFFFFFu;
    }
    two = 64 * sharers < lines;
  }
  __device__ __forceinline__ void touch(uint8_t* place) {
    const rsrc_t r = make_rsrc(base, left > 0 ? (uint64_t)left : 0);
    b2lds4(r, vo[0], 0u, place);
    if (two) b2lds4(r, vo[1], 0u, place);
    base += by;
    left -= by;
  }
};

// Operand reads: block b (32 rows) of the wave's 32 NB rows of a half, part ks of the step's four, from LDS
// addresses (32 bits; half: a constant that fits the instruction's 16-bit offset).
typedef __attribute__((address_space(3))) u32x4_t lds_u32x4_t;
template <bool ROWS, int NB = 2> struct Frags {
  uint32_t at[ROWS ? NB : 4];
  // w: which 64 rows (NB = 4: 0, all 128)
  __device__ __forceinline__ void init(const uint8_t* lds, int lane, int w) {
    const uint32_t base = (uint32_t)(uintptr_t)(lds_void_t*)lds;
    if constexpr (ROWS) {
      // group of 16 lanes: columns 16 (g & 1) .., contraction 8 (g >> 1) ..; lane l of it fetches row l / 4, four columns
      const int g = lane >> 4, l = lane & 15;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int chunk = (w * 8 + b * 4 + 2 * (g & 1) + ((l & 3) >> 1)) ^ (4 * (l >> 2));
        at[b] = base + (uint32_t)((8 * (g >> 1) + (l >> 2)) * 256 + chunk * 16 + (l & 1) * 8);
      }
    } else {
      const int l32 = lane & 31, hi = lane >> 5;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        at[ks] = base + (uint32_t)((w * 64 + l32) * 128 + 16 * ((2 * ks + hi) ^ ((l32 >> 1) & 7)));
    }
  }
  // The same reads `by` bytes further on.
  __device__ __forceinline__ Frags moved(uint32_t by) const {
    Frags f;
#pragma unroll
    for (int i = 0; i < (ROWS ? NB : 4); ++i) f.at[i] = at[i] + by;
    return f;
  }
  __device__ __forceinline__ u32x4_t read(uint32_t half, int b, int ks) const {
    if constexpr (ROWS) {
      const uint32_t p = at[b] + half + ks * 16 * 256;
      const u32x2_t x = read_tr16((const lds_s16x4_t*)p), y = read_tr16((const lds_s16x4_t*)(p + 4 * 256));
      return (u32x4_t){x[0], x[1], y[0], y[1]};
    } else {
      return *(const lds_u32x4_t*)(at[ks] + half + b * 32 * 128);
    }
  }
};

// An operand of int8 codes with the contraction as rows and a scale for each of
// those, turned into bf16(scale * code) on the way to the MFMA.  The scale differs from term to term, so it has to be
// part of a factor, and a bf16 MFMA takes factors of 8 bits: one of the two is rounded, by half a step (2^-8) at
// most.  Against fp64 the gradients are then off by 0.0023 in norm, 0.0017 of it the rounding of the results
// themselves; a second bf16 term that holds what is left would double the MFMAs (of 763 us a call at m = 4096, n = 14336, k = 4096).
// Copies (two of codes
// and one of the step's 64 scales, which every wave has for itself), reads, and the conversion.
struct Codes {
  static constexpr int kBytes = 8192;
  const uint8_t* base;
  int64_t left, ld;
  rsrc_t r, rs;
  uint32_t vo, sv;
  uint32_t at, sat;          // the wave's 32 columns, its scales

  // scales: `rows` of them.  lds, slots: addresses of the codes and of the wave's 256-byte scale slot in stage 0.
  __device__ __forceinline__ void init(const uint8_t* arr, int64_t ld_, int64_t bytes, const float* scales, int64_t rows, int tile,
                                       int first, int lane, int wave, const uint8_t* lds, const uint8_t* slot) {
    ld = ld_;
    const int64_t from = (int64_t)tile * 128 + (int64_t)first * 64 * ld;
    base = arr + from;
    left = bytes - from;
    // wave w copies rows 16 w .. + 15, eight at a time
    vo = (uint32_t)(wave * 16 + (lane >> 3)) * (uint32_t)ld + 16 * ((lane & 7) ^ (2 * ((lane >> 4) & 3)));
    rs = make_rsrc(scales, (uint64_t)rows * 4);
    sv = (uint32_t)first * 256 + lane * 4;
    const int g = lane >> 4, l = lane & 15;
    at = (uint32_t)(uintptr_t)(lds_void_t*)lds + (8 * (g >> 1) + (l >> 1)) * 128 + 32 * (wave ^ ((l >> 2) & 3)) +
         16 * (g & 1) + 8 * (l & 1);
    sat = (uint32_t)(uintptr_t)(lds_void_t*)slot + 32 * (g >> 1);
  }
  __device__ __forceinline__ void step(int s, int last) {
    r = make_rsrc(base, s < last && left > 0 ? (uint64_t)left : 0);
    base += 64 * ld;
    left -= 64 * ld;
  }
  // i = 0, 1: codes, 2: scales
  __device__ __forceinline__ void copy(int i, uint8_t* stage, uint8_t* slot, int wave) {
    if (i < 2) {
      b2lds16(r, vo + (uint32_t)i * 8 * (uint32_t)ld, 0u, stage + (wave * 16 + i * 8) * 128);
    } else {
      b2lds4(rs, sv, 0u, slot);
      sv += 256;
    }
  }
  __device__ __forceinline__ u32x2_t read(uint32_t by, int ks) const {
    return read_tr8((const lds_i32x2_t*)(at + by + ks * 16 * 128));
  }
  // scales of part ks: contraction 16 ks + 8 (lane / 32) + 4 h .. + 3
  __device__ __forceinline__ f32x4_t scales(uint32_t by, int ks, int h) const {
    typedef __attribute__((address_space(3))) f32x4_t lds_f32x4_t;
    return *(const lds_f32x4_t*)(sat + by + ks * 64 + h * 16);
  }
  // four values
  static __device__ __forceinline__ u32x2_t values(uint32_t q, f32x4_t s) {
    auto sb = [](uint32_t x, int b) { return (float)(int8_t)(x >> (8 * b)); };
    return (u32x2_t){pack_bf16(sb(q, 0) * s[0], sb(q, 1) * s[1]), pack_bf16(sb(q, 2) * s[2], sb(q, 3) * s[3])};
  }
};

// sig(g) = 1 / (1 + e^-g) as s post.  From g = -87 on post = 1, and s and everything on the way to it is in
// fp32's normal range; below, where 1 + e^g is 1, s = e^g 2^119 and post = 2^-119, which the caller multiplies by last:
// a product with a large up value or gradient can be an ordinary number where sig(g) itself has lost bits (g < -87) or
// is 0 (g < -104).  |g| s stays under 1 there (87 x 2^(119 - 125.5) at the border), so no product overflows on the way.  The exponential is
// taken 64 times larger, since it flushes results under 2^-126 and a product does not: s has 18 bits or more
// down to g = -174, where a result needs |dh u| > 2^117 to be normal itself.  The exponential's error is the
// rounding of an argument up to 126 and of log2 e (4e-6 in all), far below the bf16 rounding of the results.
struct Sigmoid {
  float s, post;
};
__device__ __forceinline__ Sigmoid sigmoid(float g) {
  const bool near = g >= -87.0f;
  const float e = __builtin_amdgcn_exp2f(near ? g * -1.4426950408889634f : __builtin_fmaf(g, 1.4426950408889634f, 125.0f));
  return {near ? __builtin_amdgcn_rcpf(1.0f + e) : e * 0x1p-6f, near ? 1.0f : 0x1p-119f};
}

// silu(g) u.
__device__ __forceinline__ float gated(float g, float u) {
  const Sigmoid sig = sigmoid(g);
  return g * sig.s * u * sig.post;
}

// Gate, up and the gradient of h to those of both, with sig = 1 / (1 + e^-g):
//   du = dh g sig,  dg = dh u (sig + g sig (1 - sig)).
// sig has no cancellation, and 1 - sig is off by less than a rounding of 1, which g (1 - sig) is added to.
__device__ __forceinline__ void gated_grad(float g, float u, float dh, float& dg, float& du) {
  const Sigmoid sig = sigmoid(g);
  const float t = g * sig.s;
  du = dh * t * sig.post;
  dg = dh * u * __builtin_fmaf(t, __builtin_fmaf(-sig.s, sig.post, 1.0f), sig.s) * sig.post;
}

// Eight bf16 values of a row at any 2-byte address (rows of an odd number of
// columns): the global memory path takes unaligned 16-byte accesses.
typedef uint32_t u32x2_a2_t __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_a2_t __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ void store8(uint16_t* row, int64_t cols, int64_t col, u32x4_t v) {
  if (col + 7 < cols) {
    *reinterpret_cast<u32x4_a2_t*>(row + col) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < cols) row[col + e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
  }
}
__device__ __forceinline__ u32x4_t load8(const uint16_t* row, int64_t cols, int64_t col) {
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (col + 7 < cols) {
    v = *reinterpret_cast<const u32x4_a2_t*>(row + col);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < cols) v[e >> 1] |= (uint32_t)row[col + e] << (16 * (e & 1));
  }
  return v;
}

// A lane of a 32 x 32 result holds columns 8 j + 4 (lane / 32) + 0..3 of one output
// row, two bf16 pairs for each j.  Swapping the upper lanes of an even j's pairs with
// the lower lanes of the odd j's gives each lane eight columns, 16 (j / 2) + 8 (lane /
// 32) + 0..7, in one 16-byte register group (and the swap is its own inverse).
__device__ __forceinline__ u32x4_t eight(u32x2_t even, u32x2_t odd) {
  const auto lo = __builtin_amdgcn_permlane32_swap(even[0], odd[0], false, false);
  const auto hi = __builtin_amdgcn_permlane32_swap(even[1], odd[1], false, false);
  return (u32x4_t){lo[0], hi[0], lo[1], hi[1]};
}

// Results of a wave's part of a tile (PB x QB blocks [P][Q] of 32 x 32) to global
// memory.  32 output rows at a time go through 4 KiB of LDS that the wave has
// for itself, so that its stores are whole 128-byte lines (pairs: 64 bytes; 32
// bytes a row straight from the registers cost 2 us a 256 x 256 tile).
//   ps: scales of the part's P rows, qs: of its rows; r0, c0: first
// output row and column; own: the wave's LDS; before: called before the first store.
//   dh: the part's values of dh (EPI_GATED_GRAD), from load_dh.
constexpr int kOwnBytes = 4096;
template <int EPI, int QB>
__device__ __forceinline__ void load_dh(const TileArgs& a, u32x4_t (&dh)[QB][2], int64_t r0, int64_t c0, int lane) {
  if (EPI != EPI_GATED_GRAD) return;
  const int l32 = lane & 31, hi = lane >> 5;
  const bool whole = r0 + 32 * QB <= a.rows && c0 + 32 <= a.cols;    // the same for all lanes
#pragma unroll
  for (int qb = 0; qb < QB; ++qb)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int64_t row = r0 + qb * 32 + l32, col = c0 + 16 * x + 8 * hi;
      if (whole) dh[qb][x] = *reinterpret_cast<const u32x4_a2_t*>(a.dh + row * a.cols + col);
      else dh[qb][x] = row < a.rows ? load8(a.dh + row * a.cols, a.cols, col) : (u32x4_t){0u, 0u, 0u, 0u};
    }
}
template <class T, int EPI, int PB, int QB, class Before>
__device__ __forceinline__ void emit(const TileArgs& a, const typename Mma<T>::Acc (&acc)[PB][QB], const u32x4_t (&dh)[QB][2], const float* ps,
                                     const float* qs, int64_t r0, int64_t c0, int lane, uint8_t* own, Before&& before) {
  constexpr int kN = kPairs<EPI> ? 1 : PB;                      // 32-column blocks of an output
  constexpr int kOuts = EPI == EPI_GATED_GRAD ? 2 : 1;
  constexpr int kRow = 64 * kN, kChunks = kRow / 16;            // bytes of a staged row, its 16-byte chunks
  constexpr int kPass = 64 / kChunks;                           // rows a store instruction covers
  const int l32 = lane & 31, hi = lane >> 5;
  const int64_t ld = kOuts * a.cols;
  auto swz = [](int r) { return kN == 2 ? (r & 7) : ((r >> 1) & 3); };
  const bool whole = r0 + 32 * QB <= a.rows && c0 + 32 * kN <= a.cols;    // the same for all lanes
#pragma unroll
  for (int qb = 0; qb < QB; ++qb) {
    const float sq = std::is_same<T, int8_t>::value ? qs[qb * 32 + l32] : 1.0f;
#pragma unroll
    for (int pb = 0; pb < kN; ++pb)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        u32x2_t d[2] = {}, o[kOuts][2];
        if (EPI == EPI_GATED_GRAD) {
          const u32x4_t t = eight((u32x2_t){dh[qb][x][0], dh[qb][x][1]}, (u32x2_t){dh[qb][x][2], dh[qb][x][3]});
          d[0] = (u32x2_t){t[0], t[1]};
          d[1] = (u32x2_t){t[2], t[3]};
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int j = 2 * x + y, n = 8 * j + 4 * hi;
          float f[kOuts][4];
          if constexpr (kPairs<EPI>) {
            const f32x4_t sg = *reinterpret_cast<const f32x4_t*>(ps + n);
            const f32x4_t su = *reinterpret_cast<const f32x4_t*>(ps + 32 + n);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float g = (float)acc[0][qb][4 * j + e] * sq * sg[e], u = (float)acc[1][qb][4 * j + e] * sq * su[e];
              if constexpr (EPI == EPI_GATED) {
                f[0][e] = gated(g, u);
              } else {
                gated_grad(g, u, (e & 1) ? hi_bf16(d[y][e >> 1]) : lo_bf16(d[y][e >> 1]), f[0][e], f[1][e]);
              }
            }
          } else if constexpr (EPI == EPI_SCALE) {
            const f32x4_t sp = *reinterpret_cast<const f32x4_t*>(ps + pb * 32 + n);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[0][e] = (float)acc[pb][qb][4 * j + e] * sq * sp[e];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[0][e] = acc[pb][qb][4 * j + e];
          }
#pragma unroll
          for (int k = 0; k < kOuts; ++k)
            o[k][y] = (u32x2_t){pack_bf16(f[k][0], f[k][1]), pack_bf16(f[k][2], f[k][3])};
        }
#pragma unroll
        for (int k = 0; k < kOuts; ++k)
          st16(own + k * 32 * kRow + l32 * kRow + 16 * ((4 * pb + 2 * x + hi) ^ swz(l32)), eight(o[k][0], o[k][1]));
      }
    if (qb == 0) before();
    __asm__ volatile("" ::: "memory");       // the wave's LDS accesses are done in order
#pragma unroll
    for (int k = 0; k < kOuts; ++k)
#pragma unroll
      for (int i = 0; i < 32 / kPass; ++i) {
        const int r = i * kPass + lane / kChunks, c = lane % kChunks;
        const u32x4_t v = ld16(own + k * 32 * kRow + r * kRow + 16 * (c ^ swz(r)));
        const int64_t row = r0 + qb * 32 + r, col = c0 + 8 * c;
        uint16_t* y = a.out + row * ld + k * a.cols;
        if (whole) *reinterpret_cast<u32x4_a2_t*>(y + col) = v;
        else if (row < a.rows) store8(y, a.cols, col, v);
      }
    __asm__ volatile("" ::: "memory");
  }
}

}  // namespace hm
