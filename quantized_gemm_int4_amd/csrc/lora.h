// Low-rank adapters of many requests: kernel arguments, workspace layout and
// the device helpers that the products (k_lora.hip) and the sums over rows
// (k_lora_grad.hip) share.
#pragma once
#include "common.h"
#include "launch.h"
#include "rows.h"

namespace hm {

constexpr int64_t kLoraMaxRows = 1 << 20;
// Most rows of a call whose blocks find their unit from the ids themselves (one
// ballot holds them all) instead of from a grouping launch: m = 48, 24 adapters
// of rank 16, k = 4096, n = 14336 12.5 us against 16.4; m = 64, 40 of rank 64, k
// = 2048, n = 7168 17.7 against 22.3.
constexpr int kLoraDirect = 64;
constexpr int kLoraPlanBlocks = 256; // most blocks of the grouping kernel
constexpr int kLoraUnit = 64;        // rows per unit of the gradient
constexpr int kTerms = 3;            // bf16 terms that carry an fp32 value of h or g into an MFMA (split4)
constexpr int kLoraCols = 256;       // output columns that an expanding block takes at a time

// Rows grouped by adapter.  A unit is up to unit_rows rows of one adapter,
// which share the loads of its matrices: units[u] = {adapter, count}, count 0
// from the last used unit on, its rows (ascending) in rows[u unit_rows ..].
// The units of an adapter are consecutive, first[e] .. first[e + 1] - 1.
struct LoraRows {
  const int32_t* units;
  const int32_t* rows;
  const int32_t* first;
  int64_t max_units;
  int unit_rows;             // 16, 32 or 64
};

struct LoraArgs {
  const uint16_t* z;         // bf16 [M][len]: the contracted rows (x, or dy)
  const uint16_t *a, *b;     // bf16 [L][rank][K], [L][N][rank]
  const float* scales;
  const int32_t* ids;
  int64_t M, N, K;
  int rank, L;
  const uint16_t* base;      // [M][cols] or null
  uint16_t* y;               // [M][cols]: the expanded rows (y, or dx)
  float* h;                  // [M][rank]: written by the forward if not null
  float* part;               // fp32 [splits][M][rank] contracted values
  int splits;
  int group, cols;           // units and columns per expanding block (one unit, or kLoraCols columns)
  LoraRows R;
};

// Sums over an adapter's rows: da = g x^T, db = dy h^T.
struct LoraGradArgs {
  const uint16_t *x, *dy;
  const float *h, *part;     // h [M][rank]; g as fp32 [splits][M][rank]
  int splits;
  int64_t M, N, K;
  int rank, L;
  uint16_t *gt, *ht;         // packed g and h, kTerms RP kLoraUnit values a unit (pack_block)
  float* sums;               // partial sums [2 chunks][rank (K + N)]
  int chunks;
  uint16_t *da, *db;
  LoraRows R;
};

// Most blocks along a contraction: an expanding block adds their sums with
// all of them in flight, in registers that it has left.
constexpr int lora_max_splits(int rp, int unit_rows, bool trans) {
  return trans ? (rp == 128 ? 4 : 8) : (unit_rows == 16 && rp == 128 ? 8 : 4);
}
// Waves of a contracting block: sixteen-row units take as many as their LDS
// images allow, each with little to do; 32-row blocks of A four, so that two
// or three blocks fit a compute unit (m = 8192, k = 4096, rank 64: 25 us, 34
// with eight).
constexpr int lora_waves(int rp, int unit_rows, bool trans) {
  return trans ? 8 : (unit_rows > 16 || rp == 128 ? 4 : (rp == 64 ? 8 : 16));
}
inline int lora_rp(int rank) { return rank <= 16 ? 16 : (rank <= 32 ? 32 : (rank <= 64 ? 64 : 128)); }

// Blocks that write an adapter's zero gradients: 16384 values each, at most 64.
inline int lora_zero_parts(int rank, int64_t K, int64_t N) {
  const int64_t parts = (rank * (K + N) + 16383) / 16384;
  return (int)(parts < 64 ? parts : 64);
}

// Grouping of M rows by adapter id (ids outside [0, L) are left out).
hipError_t launch_lora_plan(const int32_t* ids, int64_t M, int L, int unit_rows, int64_t max_units, int32_t* units,
                            int32_t* rows, int32_t* first, hipStream_t st);
// part = scale * (A z) or, trans, scale * (B^T z).  direct: units found from
// the ids by every block (M <= kLoraDirect, 16 rows a unit).
hipError_t launch_lora_shrink(const LoraArgs& g, bool direct, bool trans, hipStream_t st);
// y = base + B h.
hipError_t launch_lora_expand(const LoraArgs& g, bool direct, hipStream_t st);
// both forward products in one launch (M <= 16, rank <= 64)
hipError_t launch_lora_small(const LoraArgs& g, int parts, hipStream_t st);
// packed g and h, zeros for adapters without rows, and (g.y not null) y = base + A^T g
hipError_t launch_lora_dx(const LoraArgs& g, const LoraGradArgs& o, hipStream_t st);
hipError_t launch_lora_outer(const LoraGradArgs& g, hipStream_t st);
hipError_t launch_lora_sums(const LoraGradArgs& g, hipStream_t st);

#ifdef __HIPCC__
template <int N> struct Int { static constexpr int value = N; };

// fp32 pair -> four pairs of bf16 terms.  The first kTerms carry v: each is the
// leading eight bits, cut off, of what the ones before it leave, 24 in all (of
// values of 2^-102 and more).  A term is multiplied by values that may be
// infinite, so all four have v's sign and none is 0 unless v is: where nothing
// is left, and as the fourth, stands 2^-32 v, too small to change a sum.  An
// infinite or NaN v has itself in all four.
__device__ __forceinline__ void split4(float a, float b, uint32_t t[4]) {
  float v[2] = {a, b};
  const float e[2] = {a * 0x1p-32f, b * 0x1p-32f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t p[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      p[j] = __float_as_uint(i < kTerms && __builtin_fabsf(v[j]) > 0.f ? v[j] : e[j]);
      v[j] -= __uint_as_float(__float_as_uint(v[j]) & 0xffff0000u);
    }
    t[i] = __builtin_amdgcn_perm(p[1], p[0], 0x07060302u);
  }
}

// Keeps the loads written before this point before it (the compiler would
// otherwise move each next to its use, one round trip to memory per load).
__device__ __forceinline__ void loads_first() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Words of eight rows of W (1, 2, 4, 8) neighbouring 16-bit columns, and
// their transpose: value i of column j's operand is row i.
template <int W> struct Cols8 {
  uint32_t w[8][(W + 1) / 2];
  __device__ __forceinline__ void load(const uint16_t* p, int64_t stride, int ok) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint16_t* r = p + i * stride;
      if constexpr (W == 8) {
        const u32x4_t v = i < ok ? ld16(r) : (u32x4_t){0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < 4; ++k) w[i][k] = v[k];
      } else if constexpr (W == 4) {
        const u32x2_t v = i < ok ? *reinterpret_cast<const u32x2_t*>(r) : (u32x2_t){0u, 0u};
        w[i][0] = v[0];
        w[i][1] = v[1];
      } else if constexpr (W == 2) {
        w[i][0] = i < ok ? *reinterpret_cast<const uint32_t*>(r) : 0u;
      } else {
        w[i][0] = i < ok ? *r : 0u;
      }
    }
  }
  __device__ __forceinline__ u32x4_t operand(int j) const {
    u32x4_t o;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = __builtin_amdgcn_perm(w[2 * k + 1][j >> 1], w[2 * k][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
    return o;
  }
};
#endif

}  // namespace hm
