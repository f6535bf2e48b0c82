// Parts of the stable counting sorts of ids by expert or adapter (k_moe.hip,
// k_rows.hip, k_lora.hip): a block's scan, and a block's placing of a range.
#pragma once
#include "common.h"

namespace hm {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;

// Inclusive scan of one value per thread over the first 512 threads of a
// block (8 waves).  `wsum` is 8 ints of shared scratch.  Must be reached by
// every thread of the block.
__device__ inline int block_scan512(int v, int* wsum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int off = 1; off < 64; off <<= 1) {
    const int u = __shfl_up(v, off, 64);
    if (lane >= off) v += u;
  }
  if (lane == 63 && wave < 8) wsum[wave] = v;
  __syncthreads();
  int pre = 0;
  for (int w = 0; w < wave && w < 8; ++w) pre += wsum[w];
  __syncthreads();
  return v + pre;
}

// Places the pairs of [lo, hi) stably: wave w owns the contiguous subrange
// [lo + w*chunk, ...), its per-expert base positions are base[e] plus the
// counts of earlier waves, and inside a wave each batch of 64 pairs is ranked
// in lane order with ballot matching.  hist is the block's [16][512] LDS
// array (zeroed here); base[e] (LDS) is the first position of this range's
// pairs of expert e.  POS: also the inverse, positions[p] (-1 for a dropped
// pair).  Must be reached by every thread of the block.
template <bool POS>
__device__ inline void sort_range(const int32_t* __restrict__ ids, int64_t lo, int64_t hi, int E, const int* base,
                           int (*hist)[512], int32_t* __restrict__ sorted_pairs, int32_t* __restrict__ positions) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < kSortWaves * 512; i += kSortThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  const int64_t chunk = (hi - lo + kSortWaves - 1) / kSortWaves;
  const int64_t beg = lo + wave * chunk;
  const int64_t end = (beg + chunk < hi) ? beg + chunk : hi;
  for (int64_t b = beg; b < end; b += 64) {
    const int64_t p = b + lane;
    if (p < end) {
      const int e = ids[p];
      if (e >= 0 && e < E) atomicAdd(&hist[wave][e], 1);
    }
  }
  __syncthreads();
  if (tid < E) {
    int run = base[tid];
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = hist[w][tid];
      hist[w][tid] = run;
      run += c;
    }
  }
  __syncthreads();
  int nbits = 0;
  while ((1 << nbits) < E) ++nbits;
  const uint64_t lt = (lane == 0) ? 0ull : (~0ull >> (64 - lane));
  for (int64_t b = beg; b < end; b += 64) {
    const int64_t p = b + lane;
    int e = -1;
    if (p < end) e = ids[p];
    const bool valid = (e >= 0 && e < E);
    uint64_t m = __ballot(valid);
    for (int bit = 0; bit < nbits; ++bit) {
      const uint64_t x = __ballot(valid && ((e >> bit) & 1));
      m &= ((e >> bit) & 1) ? x : ~x;
    }
    if (valid) {
      const int rank = __popcll(m & lt);
      const int pos = hist[wave][e] + rank;
      sorted_pairs[pos] = (int32_t)p;
      if (POS) positions[p] = pos;
    } else if (POS && p < end) {
      positions[p] = -1;
    }
    __builtin_amdgcn_wave_barrier();
    if (valid && __popcll(m & lt) == 0) hist[wave][e] += __popcll(m);
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace hm
