// Token rows to and from expert order (tokens split per expert:
// aihaber.org article on Humming, "what problem does it solve"; ywsung.com
// note "How vLLM Humming computes 4 bits", section on one token vs many
// tokens).  positions[p] is the expert-ordered row of pair p = t topk + j:
//   dispatch       xs[positions[p]] = x[p / topk]
//   collect        out[t] = sum_j w[t][j] ys[positions[t topk + j]]
//   its gradient   dys[positions[p]] = w[p] dout[p / topk],
//                  dw[p] = sum_c dout[p / topk][c] ys[positions[p]][c]
// All three only move bf16 rows: every row of the token side is read (or
// written) once and every row of the expert side once, so they are bound by
// HBM, and calls of few tokens by their launches and round trips.  Measured at
// n = 7168, topk = 8 (a 1 GiB device copy runs at 5.1 TB/s, read and written
// bytes together): dispatch t = 8192 205 us, 5.2 TB/s; collect and the
// dispatch's gradient t = 4096 103 us, 5.1 TB/s, t = 8192 205 us; collect's
// gradient t = 4096 199 us, 5.0 TB/s; t = 64 dispatch 5.9 us, collect 4.0 us.
#include "common.h"
#include "launch.h"
#include "rows.h"
#include "sort.h"

namespace hm {

constexpr int kPairs = 8;      // pairs of a token whose rows are in flight together

// The expert-ordered rows of pairs j0 .. j0 + kPairs - 1 of token t (-1: no
// row), read by one lane each and handed to the wave.
__device__ __forceinline__ void token_rows(const int32_t* __restrict__ positions, int64_t t, int topk, int j0, int64_t P,
                                           int64_t pos[kPairs]) {
  const int lane = threadIdx.x & 63;
  int p = -1;
  if (lane < kPairs && j0 + lane < topk) p = positions[t * topk + j0 + lane];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const int v = __builtin_amdgcn_readlane(p, j);
    pos[j] = v < P ? v : -1;
  }
}

// A wave per (token, 512 columns): the chunk is read once and written to each
// of the token's expert rows.
__global__ void __launch_bounds__(256)
k_dispatch_rows(const uint16_t* __restrict__ x, const int32_t* __restrict__ positions, int64_t t_count, int topk,
                int64_t n, int segs, uint16_t* __restrict__ xs) {
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t = w / segs, c = 512 * (w - t * segs) + 8 * (threadIdx.x & 63);
  if (t >= t_count) return;
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (c < n) v = ld8_tail(x + t * n, c, n);
  for (int j0 = 0; j0 < topk; j0 += kPairs) {
    int64_t pos[kPairs];
    token_rows(positions, t, topk, j0, t_count * topk, pos);
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
      if (pos[j] >= 0 && c < n) st8_tail(xs + pos[j] * n, c, n, v);
  }
}

// A wave per (token, 512 columns): the fp32 sum over the token's rows in
// ascending j, eight rows' loads in flight.
template <bool W>
__global__ void __launch_bounds__(256)
k_collect(const uint16_t* __restrict__ ys, const float* __restrict__ w, const int32_t* __restrict__ positions,
          int64_t t_count, int topk, int64_t n, int segs, uint16_t* __restrict__ out) {
  const int64_t wi = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t = wi / segs, c = 512 * (wi - t * segs) + 8 * (threadIdx.x & 63);
  if (t >= t_count) return;
  const int lane = threadIdx.x & 63;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < topk; j0 += kPairs) {
    int64_t pos[kPairs];
    float wl = 1.0f;
    if (W && lane < kPairs && j0 + lane < topk) wl = w[t * topk + j0 + lane];
    token_rows(positions, t, topk, j0, t_count * topk, pos);
    u32x4_t v[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
      if (pos[j] >= 0 && c < n) v[j] = ld8_tail(ys + pos[j] * n, c, n);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      if (pos[j] < 0) continue;
      const float wj = W ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wl), j)) : 1.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[2 * e] = fmaf(wj, lo_bf16(v[j][e]), acc[2 * e]);
        acc[2 * e + 1] = fmaf(wj, hi_bf16(v[j][e]), acc[2 * e + 1]);
      }
    }
  }
  if (c < n)
    st8_tail(out + t * n, c, n, (u32x4_t){pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                                          pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7])});
}

// One block per token, eight pairs at a time: dout is read once for them, and
// dw is a reduction in a fixed order.  ys and dys may be the same rows: each
// chunk is read before the thread that read it writes it.
__global__ void __launch_bounds__(512)
k_collect_grad(const uint16_t* __restrict__ dout, const uint16_t* ys, const float* __restrict__ w,
               const int32_t* __restrict__ positions, int64_t t_count, int topk, int64_t n, uint16_t* dys,
               float* __restrict__ dw) {
  __shared__ float red[8][kPairs];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int j0 = 0; j0 < topk; j0 += kPairs) {
    int64_t pos[kPairs];
    float wl = 0.f;
    if (lane < kPairs && j0 + lane < topk) wl = w[t * topk + j0 + lane];
    token_rows(positions, t, topk, j0, t_count * topk, pos);
    float s[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) s[j] = 0.f;
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < n; c += 8 * (int64_t)blockDim.x) {
      const u32x4_t d = ld8_tail(dout + t * n, c, n);
      u32x4_t y[kPairs];
#pragma unroll
      for (int j = 0; j < kPairs; ++j)
        if (pos[j] >= 0) y[j] = ld8_tail(ys + pos[j] * n, c, n);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        if (pos[j] < 0) continue;
        const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wl), j));
        u32x4_t o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[j] = fmaf(lo_bf16(d[e]), lo_bf16(y[j][e]), s[j]);
          s[j] = fmaf(hi_bf16(d[e]), hi_bf16(y[j][e]), s[j]);
          o[e] = pack_bf16(wj * lo_bf16(d[e]), wj * hi_bf16(d[e]));
        }
        st8_tail(dys + pos[j] * n, c, n, o);
      }
    }
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      if (j0 + j >= topk) break;
      for (int off = 32; off >= 1; off >>= 1) s[j] += __shfl_xor(s[j], off, 64);
      if (lane == 0) red[wave][j] = s[j];
    }
    __syncthreads();
    if ((int)threadIdx.x < kPairs && j0 + (int)threadIdx.x < topk) {
      float v = 0.f;
      for (int k = 0; k < (int)blockDim.x / 64; ++k) v += red[k][threadIdx.x];
      dw[t * topk + j0 + threadIdx.x] = v;
    }
    __syncthreads();
  }
}

// counts and offsets of E <= 512 experts from their totals; every thread of a
// block of 512 or more.
__device__ __forceinline__ int write_offsets(int total, int E, int* wsum, int32_t* __restrict__ counts,
                                             int32_t* __restrict__ offsets, bool out) {
  const int tid = threadIdx.x;
  const int end = block_scan512(tid < 512 ? total : 0, wsum);
  if (out && tid < E) {
    counts[tid] = total;
    offsets[tid] = end - total;
    if (tid == E - 1) offsets[E] = end;
  }
  return end - total;
}

// The stable expert sort of hm_moe_sort with its inverse, in one launch (up to
// kSortDispatch pairs): every block counts all ids (and those before its
// own 1024), as k_lora_plan does.
__global__ void __launch_bounds__(kSortThreads)
k_dispatch_sort(const int32_t* __restrict__ ids, int64_t P, int E, int32_t* __restrict__ counts,
                int32_t* __restrict__ offsets, int32_t* __restrict__ sorted_pairs, int32_t* __restrict__ positions) {
  __shared__ int hist[kSortWaves][512];
  __shared__ int before[512], after[512], base[512];
  __shared__ int wsum[8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t lo = (int64_t)blockIdx.x * kSortThreads;
  const int own = lo + tid < P ? ids[lo + tid] : -1;
  for (int i = tid; i < 512; i += kSortThreads) before[i] = after[i] = 0;
  for (int i = tid; i < kSortWaves * 512; i += kSortThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  for (int64_t p0 = 0; p0 < P; p0 += 8 * kSortThreads) {
    int id[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t p = p0 + i * kSortThreads + tid;
      id[i] = p < P ? ids[p] : -1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (id[i] >= 0 && id[i] < E) atomicAdd(p0 + i * kSortThreads < lo ? &before[id[i]] : &after[id[i]], 1);
  }
  __syncthreads();
  const int total = tid < 512 ? before[tid] + after[tid] : 0;
  const int first = write_offsets(total, E, wsum, counts, offsets, blockIdx.x == 0);
  if (tid < 512) base[tid] = first + before[tid];
  const bool ok = own >= 0 && own < E;
  int nbits = 0;
  while ((1 << nbits) < E) ++nbits;
  uint64_t m = __ballot(ok);
  for (int bit = 0; bit < nbits; ++bit) {
    const uint64_t x = __ballot(ok && ((own >> bit) & 1));
    m &= ((own >> bit) & 1) ? x : ~x;
  }
  const int rank = __popcll(m & (lane ? (~0ull >> (64 - lane)) : 0ull));
  if (ok && rank == 0) hist[wave][own] = __popcll(m);
  __syncthreads();
  int at = -1;
  if (ok) {
    at = base[own] + rank;
    for (int w = 0; w < wave; ++w) at += hist[w][own];
    sorted_pairs[at] = (int32_t)(lo + tid);
  }
  if (lo + tid < P) positions[lo + tid] = at;
}

// Sort and rows of up to kSmallPairs pairs in one launch.  grid (column
// parts, t + 1): the block of a token finds its pairs' places by counting the
// ids before them; the block behind the last token writes counts and offsets.
__global__ void __launch_bounds__(512)
k_dispatch_small(const uint16_t* __restrict__ x, const int32_t* __restrict__ ids, int64_t t_count, int topk, int E,
                 int64_t n, uint16_t* __restrict__ xs, int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                 int32_t* __restrict__ sorted_pairs, int32_t* __restrict__ positions) {
  __shared__ int hist[512];
  __shared__ int wsum[8];
  __shared__ int places[8][kPairs];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, P = (int)(t_count * topk);
  int id[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    id[i] = tid + 512 * i < P ? ids[tid + 512 * i] : -1;
    if (id[i] >= E) id[i] = -1;
  }
  const int64_t t = blockIdx.y;
  if (t == t_count) {
    if (blockIdx.x) return;
    hist[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (id[i] >= 0) atomicAdd(&hist[id[i]], 1);
    __syncthreads();
    write_offsets(hist[tid], E, wsum, counts, offsets, true);
    return;
  }
  const int64_t chunks = (n + 7) / 8, c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
  for (int j0 = 0; j0 < topk; j0 += kPairs) {
    int e[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const int p = (int)(t * topk) + j0 + j;
      e[j] = j0 + j < topk ? ids[p] : -1;
      if (e[j] >= E) e[j] = -1;
      int c = 0;                                              // valid pairs of lower experts, or of this one and before p
#pragma unroll
      for (int i = 0; i < 2; ++i)
        c += __popcll(__ballot(id[i] >= 0 && (id[i] < e[j] || (id[i] == e[j] && tid + 512 * i < p))));
      if (lane == 0) places[wave][j] = c;
    }
    __syncthreads();
    int pos[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      int c = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) c += places[k][j];
      pos[j] = e[j] >= 0 ? c : -1;
    }
    if (blockIdx.x == 0 && tid < kPairs && j0 + tid < topk) {
      int at = -1;
#pragma unroll
      for (int j = 0; j < kPairs; ++j)
        if (j == tid) at = pos[j];
      const int p = (int)(t * topk) + j0 + tid;
      positions[p] = at;
      if (at >= 0) sorted_pairs[at] = p;
    }
    for (int64_t ch = c0 + tid; ch < c1; ch += 512) {
      const u32x4_t v = ld8_tail(x + t * n, 8 * ch, n);
#pragma unroll
      for (int j = 0; j < kPairs; ++j)
        if (pos[j] >= 0) st8_tail(xs + (int64_t)pos[j] * n, 8 * ch, n, v);
    }
    __syncthreads();
  }
}

hipError_t launch_dispatch_small(const uint16_t* x, const int32_t* ids, int64_t t, int topk, int E, int64_t n,
                                 uint16_t* xs, int32_t* counts, int32_t* offsets, int32_t* sorted_pairs,
                                 int32_t* positions, hipStream_t st) {
  // parts of at least 128 chunks (64 KB of rows at topk = 8), about 256 blocks
  const int64_t most = ((n + 7) / 8 + 127) / 128, want = (256 + t - 1) / t;
  const dim3 grid((unsigned)(want < most ? want : most), (unsigned)(t + 1));
  hipLaunchKernelGGL(k_dispatch_small, grid, dim3(512), 0, st, x, ids, t, topk, E, n, xs, counts, offsets, sorted_pairs,
                     positions);
  return hipGetLastError();
}

hipError_t launch_dispatch_sort(const int32_t* ids, int64_t P, int E, int32_t* counts, int32_t* offsets,
                                int32_t* sorted_pairs, int32_t* positions, hipStream_t st) {
  hipLaunchKernelGGL(k_dispatch_sort, dim3((unsigned)((P + kSortThreads - 1) / kSortThreads)), dim3(kSortThreads), 0, st,
                     ids, P, E, counts, offsets, sorted_pairs, positions);
  return hipGetLastError();
}

// blocks of four waves, a wave per (token, 512 columns)
static dim3 wave_grid(int64_t t, int64_t n, int* segs) {
  *segs = (int)((n + 511) / 512);
  return dim3((unsigned)((t * *segs + 3) / 4));
}

hipError_t launch_dispatch_rows(const uint16_t* x, const int32_t* positions, int64_t t, int topk, int64_t n,
                                uint16_t* xs, hipStream_t st) {
  int segs;
  const dim3 grid = wave_grid(t, n, &segs);
  hipLaunchKernelGGL(k_dispatch_rows, grid, dim3(256), 0, st, x, positions, t, topk, n, segs, xs);
  return hipGetLastError();
}

hipError_t launch_collect(const uint16_t* ys, const float* w, const int32_t* positions, int64_t t, int topk,
                          int64_t n, uint16_t* out, hipStream_t st) {
  int segs;
  const dim3 grid = wave_grid(t, n, &segs);
  if (w) hipLaunchKernelGGL(k_collect<true>, grid, dim3(256), 0, st, ys, w, positions, t, topk, n, segs, out);
  else hipLaunchKernelGGL(k_collect<false>, grid, dim3(256), 0, st, ys, w, positions, t, topk, n, segs, out);
  return hipGetLastError();
}

hipError_t launch_collect_grad(const uint16_t* dout, const uint16_t* ys, const float* w, const int32_t* positions,
                               int64_t t, int topk, int64_t n, uint16_t* dys, float* dw, hipStream_t st) {
  // A block's threads take 8 columns each, so 512 of them would idle below n = 4096, or wait for little work: topk = 8,
  // n = 2048, t = 4096 49 us with 256 threads, 61 with 512 (n = 1024: 29, 44); n = 7168, t = 64 11.2 with 256, 9.2 with
  // 512, t = 4096 208 and 206.  A launch stays under 2^32 threads: from 2^23 tokens on 256, whatever n.
  const int threads = n <= 2048 || t >= (1 << 23) ? 256 : 512;
  hipLaunchKernelGGL(k_collect_grad, dim3((unsigned)t), dim3(threads), 0, st, dout, ys, w, positions, t, topk, n, dys,
                     dw);
  return hipGetLastError();
}

}  // namespace hm
