// Launchers of the operators on rows in expert order (k_rows.hip) and of the
// low-rank adapters (k_lora.hip, k_lora_grad.hip), and what their planners
// share with them.
#pragma once
#include "common.h"
#include "launch.h"

namespace hm {

// bf16 rows of any length: eight values at any 2-byte address (one 16-byte
// access; unaligned ones are legal for global memory on gfx950).
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
__device__ __forceinline__ u32x4_t ld8(const uint16_t* p) {
  return *reinterpret_cast<const u32x4_any_t*>(p);
}
__device__ __forceinline__ void st8(uint16_t* p, u32x4_t v) { *reinterpret_cast<u32x4_any_t*>(p) = v; }

// Values c .. c + 7 of a row of n (zeros from n on); c < n.
__device__ __forceinline__ u32x4_t ld8_tail(const uint16_t* row, int64_t c, int64_t n) {
  if (c + 8 <= n) return ld8(row + c);
  u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < n) v[e >> 1] |= (uint32_t)row[c + e] << (16 * (e & 1));
  return v;
}
__device__ __forceinline__ void st8_tail(uint16_t* row, int64_t c, int64_t n, u32x4_t v) {
  if (c + 8 <= n) {
    st8(row + c, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < n) row[c + e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
}

// The same four values at a time.
typedef u32x2_t u32x2_any_t __attribute__((aligned(2)));
__device__ __forceinline__ u32x2_t ld4_tail(const uint16_t* row, int64_t c, int64_t n) {
  if (c + 4 <= n) return *reinterpret_cast<const u32x2_any_t*>(row + c);
  u32x2_t v = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < n) v[e >> 1] |= (uint32_t)row[c + e] << (16 * (e & 1));
  return v;
}
__device__ __forceinline__ void st4_tail(uint16_t* row, int64_t c, int64_t n, u32x2_t v) {
  if (c + 4 <= n) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x2_any_t*>(row + c));
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < n) row[c + e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
}

// Pairs that are sorted and moved in one launch, each token's block counting
// all ids for itself (two a thread): t = 64, topk = 8, n = 7168 5.9 us against
// 8.6 with a sort of its own.
constexpr int64_t kSmallPairs = 1024;
// Pairs that are sorted in one launch, each block counting all ids, where a
// chunked sort counts and places in two: with rows of n = 2048, topk = 8, 2048
// pairs 9.1 us against 11.7, 8192 14.0 against 16.6, 32768 33.6 against 34.3,
// and 65536 65.4 against 63.0; of n = 7168, 8192 pairs 27.9 against 30.5, 65536
// 208 against 204.
constexpr int64_t kSortDispatch = 32768;
hipError_t launch_dispatch_small(const uint16_t* x, const int32_t* ids, int64_t t, int topk, int E, int64_t n,
                                 uint16_t* xs, int32_t* counts, int32_t* offsets, int32_t* sorted_pairs,
                                 int32_t* positions, hipStream_t st);
hipError_t launch_dispatch_sort(const int32_t* ids, int64_t P, int E, int32_t* counts, int32_t* offsets,
                                int32_t* sorted_pairs, int32_t* positions, hipStream_t st);
// xs[positions[p]] = x[p / topk] for positions in [0, t topk)
hipError_t launch_dispatch_rows(const uint16_t* x, const int32_t* positions, int64_t t, int topk, int64_t n,
                                uint16_t* xs, hipStream_t st);
// out[t] = sum_j w[t][j] ys[positions[t][j]] (w null: 1)
hipError_t launch_collect(const uint16_t* ys, const float* w, const int32_t* positions, int64_t t, int topk,
                          int64_t n, uint16_t* out, hipStream_t st);
hipError_t launch_collect_grad(const uint16_t* dout, const uint16_t* ys, const float* w, const int32_t* positions,
                               int64_t t, int topk, int64_t n, uint16_t* dys, float* dw, hipStream_t st);

}  // namespace hm
