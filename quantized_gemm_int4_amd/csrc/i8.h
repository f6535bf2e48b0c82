// Linear layers in 8-bit integers (one fp32 scale per token and per output
// channel), their gated block and gradients: internal launchers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hm {

// What a tile kernel does with its sums (row q of the output, column p):
enum I8Epi : int {
  EPI_SCALE = 0,       // bf16(acc * qs[q] * ps[p]), integer sums
  EPI_GATED = 1,       // P rows are gate / up pairs: bf16(silu(g) * u)
  EPI_GATED_GRAD = 2,  // the same pairs and dh: bf16(dg), bf16(du)
  EPI_ROUND = 3        // bf16(acc), fp32 sums of bf16 products
};

// One product O[q][p] = sum_c Q[q][c] P[p][c].  An operand is held either with
// the contraction along its rows (c contiguous) or with the contraction as its
// rows (p or q contiguous, bf16 only); which one is the kernel's template.
struct TileArgs {
  const uint8_t* p;       // operand of the output's columns; gated: gate rows 0..d-1, up rows d..2d-1
  int64_t p_ld, p_bytes;  // bytes between its rows, bytes of the array (gated: of one half)
  const uint8_t* q;       // operand of the output's rows
  int64_t q_ld, q_bytes;
  int64_t rows, cols;     // of the output (gated: cols = d, of h or of each of dg and du)
  int64_t kbytes;         // contraction length in bytes of one element row (steps of 128)
  const float* ps;        // scales (integer products; tiles of 128 of a gradient: of the `terms` rows of P)
  const float* qs;
  int64_t terms;
  const uint16_t* dh;     // EPI_GATED_GRAD: [rows][cols]
  uint16_t* out;          // bf16 [rows][cols] (EPI_GATED_GRAD: [rows][2 cols])
};

enum I8Kind : int { I8_FORWARD = 0, I8_GATED = 1, I8_GATED_GRAD = 2, I8_DX = 3, I8_DW = 4 };

// 128 x 128 output tiles.  Tiles from number `full` on are cut along the
// contraction into `cut` parts of `per` steps of 128 bytes, whose sums go to
// part [(tile - full) * cut][128][128], 4 bytes each.
constexpr int kI8Tile = 128;
struct TilePlan {
  int tiles_p, tiles_q;
  int full, cut, per;
  int two;                   // two blocks a compute unit, of two stages each
  int codes;                 // gradients: P is int8 codes with scales ps, not their bf16 copy
  void* part;
};
hipError_t launch_i8_tile(const TileArgs& a, const TilePlan& pl, int kind, hipStream_t st);
// 256 x 256 output tiles: blocks of four waves, one a compute unit
constexpr int kI8Big = 256;
hipError_t launch_i8_big(const TileArgs& a, int kind, hipStream_t st);

// Products (not I8_DX, I8_DW) of up to kI8Few rows: blocks of a few weight rows against groups of up to 128 rows of x.
constexpr int64_t kI8Few = 1024;
struct FewPlan {
  int groups, rows;          // groups, rows of each (but the last), a multiple of 16
  int nb;                    // blocks of 16 weight rows (pairs: of gate and up) a block takes, 1 .. 4, pairs two or four
};
// The most blocks of weights a block takes: more share its rows of x, of which few rows have too little to gain
// (k = 6656, m = 11, n = 8256: three 13.6 us, one 13.8).
constexpr int i8_few_most(int row_blocks, bool pairs) { return row_blocks >= 4 ? 4 : pairs || row_blocks == 1 ? 2 : 3; }
hipError_t launch_i8_few(const TileArgs& a, const FewPlan& p, int kind, hipStream_t st);

// I8_DX for few rows, P as codes: blocks of 64 columns against groups of `rows` rows (32, 64 or 128)
hipError_t launch_i8_few_dx(const TileArgs& a, int rows, hipStream_t st);

// bf16 rows -> int8 codes and fp32 scales
hipError_t launch_i8_quant_rows(const uint16_t* x, int64_t m, int64_t k, int8_t* x8, float* s, hipStream_t st);
// Copies for a gradient: two arrays of int8 rows of 16 kc codes -> bf16(scale * code), none where rows = 0, and m rows
// of n bf16 values -> rows of 8 nc >= n, zeros behind, none where nc = 0.
struct I8Copies {
  const int8_t* q[2];
  const float* s[2];
  uint16_t* out[2];
  int64_t rows[2], kc;
  const uint16_t* dy;
  uint16_t* pad;
  int64_t m, n, nc;
};
hipError_t launch_i8_copies(const I8Copies& c, hipStream_t st);

}  // namespace hm
