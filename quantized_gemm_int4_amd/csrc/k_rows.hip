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
// HBM.
#include "common.h"
#include "launch.h"
#include "rows.h"

namespace hm {

// One block per token, 16-byte chunks over its threads: the token's chunk is
// read once and written to each of its expert rows.
__global__ void __launch_bounds__(256)
k_dispatch_rows(const uint16_t* __restrict__ x, const int32_t* __restrict__ positions, int64_t P, int topk, int64_t n,
                uint16_t* __restrict__ xs) {
  const int64_t t = blockIdx.x;
  const int32_t* pos = positions + t * topk;
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < n; c += 8 * 256) {
    const u32x4_t v = ld8_tail(x + t * n, c, n);
    for (int j = 0; j < topk; ++j) {
      const int64_t p = pos[j];
      if (p >= 0 && p < P) st8_tail(xs + p * n, c, n, v);
    }
  }
}

// One block per token: the fp32 sum over its rows in ascending j.
template <bool W>
__global__ void __launch_bounds__(256)
k_collect(const uint16_t* __restrict__ ys, const float* __restrict__ w, const int32_t* __restrict__ positions, int64_t P,
          int topk, int64_t n, uint16_t* __restrict__ out) {
  const int64_t t = blockIdx.x;
  const int32_t* pos = positions + t * topk;
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < n; c += 8 * 256) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < topk; ++j) {
      const int64_t p = pos[j];
      if (p < 0 || p >= P) continue;
      const float wj = W ? w[t * topk + j] : 1.0f;
      const u32x4_t v = ld8_tail(ys + p * n, c, n);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[2 * e] = fmaf(wj, lo_bf16(v[e]), acc[2 * e]);
        acc[2 * e + 1] = fmaf(wj, hi_bf16(v[e]), acc[2 * e + 1]);
      }
    }
    st8_tail(out + t * n, c, n, (u32x4_t){pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                                          pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7])});
  }
}

// One block per token and pair: dw is a block reduction in a fixed order.
// ys and dys may be the same rows: each chunk is read before the thread that
// read it writes it.
__global__ void __launch_bounds__(256)
k_collect_grad(const uint16_t* __restrict__ dout, const uint16_t* ys, const float* __restrict__ w,
               const int32_t* __restrict__ positions, int64_t P, int topk, int64_t n, uint16_t* dys,
               float* __restrict__ dw) {
  __shared__ float red[4];
  const int64_t t = blockIdx.x;
  for (int j = 0; j < topk; ++j) {
    const int64_t p = positions[t * topk + j];
    float s = 0.f;
    if (p >= 0 && p < P) {
      const float wj = w[t * topk + j];
      for (int64_t c = 8 * (int64_t)threadIdx.x; c < n; c += 8 * 256) {
        const u32x4_t d = ld8_tail(dout + t * n, c, n), y = ld8_tail(ys + p * n, c, n);
        u32x4_t o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s = fmaf(lo_bf16(d[e]), lo_bf16(y[e]), s);
          s = fmaf(hi_bf16(d[e]), hi_bf16(y[e]), s);
          o[e] = pack_bf16(wj * lo_bf16(d[e]), wj * hi_bf16(d[e]));
        }
        st8_tail(dys + p * n, c, n, o);
      }
    }
    for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) dw[t * topk + j] = (red[0] + red[1]) + (red[2] + red[3]);
    __syncthreads();
  }
}

hipError_t launch_dispatch_rows(const uint16_t* x, const int32_t* positions, int64_t t, int topk, int64_t n,
                                uint16_t* xs, hipStream_t st) {
  hipLaunchKernelGGL(k_dispatch_rows, dim3((unsigned)t), dim3(256), 0, st, x, positions, t * topk, topk, n, xs);
  return hipGetLastError();
}

hipError_t launch_collect(const uint16_t* ys, const float* w, const int32_t* positions, int64_t t, int topk,
                          int64_t n, uint16_t* out, hipStream_t st) {
  if (w) hipLaunchKernelGGL(k_collect<true>, dim3((unsigned)t), dim3(256), 0, st, ys, w, positions, t * topk, topk, n, out);
  else hipLaunchKernelGGL(k_collect<false>, dim3((unsigned)t), dim3(256), 0, st, ys, w, positions, t * topk, topk, n, out);
  return hipGetLastError();
}

hipError_t launch_collect_grad(const uint16_t* dout, const uint16_t* ys, const float* w, const int32_t* positions,
                               int64_t t, int topk, int64_t n, uint16_t* dys, float* dw, hipStream_t st) {
  hipLaunchKernelGGL(k_collect_grad, dim3((unsigned)t), dim3(256), 0, st, dout, ys, w, positions, t * topk, topk, n,
                     dys, dw);
  return hipGetLastError();
}

}  // namespace hm
