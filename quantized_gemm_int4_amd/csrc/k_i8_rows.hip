// Rows of the 8-bit integer layers: quantization per token (the codes that the
// product multiplies, and what a training step keeps of its activations), the
// bf16 form of 8-bit rows for the gradients, and padded copies of odd rows.
#include <hip/hip_runtime.h>

#include "common.h"
#include "i8.h"

namespace hm {

namespace {

// The code of x in a row with largest magnitude amax is the whole number
// nearest to v = 127 x / amax, ties to even.  v is a ratio of whole numbers:
// with 8-bit significands X and A, v = 127 X / (A 2^c), and for a tie j + 1/2 that v
// does not meet, |v - (j + 1/2)| >= 1 / (A 2^c) = v / (127 X) > v 2^-15.  The fp32
// product x (127 / amax) has two roundings, at most 2^-23 of v.  So rounding it to 19
// significant bits (the integer add and mask; it moves a value by at most 2^-19
// of itself) brings every tie to its exact value and moves nothing else across
// one; the second rounding, to whole numbers, then sees what the ratio itself
// would give.
struct Coder {
  float inv;                 // 127 / (amax pre)
  float pre;                 // a power of two that keeps 127 / (amax pre) and the products in range
  __device__ __forceinline__ int code(float x) const {
    const float t = (x * pre) * inv;
    return (int)__builtin_rintf(__uint_as_float((__float_as_uint(t) + 16u) & ~31u));
  }
};

__device__ __forceinline__ Coder coder_of(float amax) {
  // by 2^100 for tiny rows (exact), by 2^-30 for huge ones (exact for every value whose code is not 0)
  Coder c;
  c.pre = amax < 0x1p-100f ? 0x1p100f : (amax > 0x1p100f ? 0x1p-30f : 1.0f);
  c.inv = __fdiv_rn(127.0f, amax * c.pre);
  return c;
}

// Largest magnitude of bf16 pairs as bits: magnitudes order like their bit
// patterns, and infinities and NaN come out on top.
__device__ __forceinline__ uint32_t amax_bits(uint32_t m, uint32_t pair) {
  const uint32_t lo = (pair << 16) & 0x7FFF0000u, hi = pair & 0x7FFF0000u;
  return max(m, max(lo, hi));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  for (int off = 32; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
  return v;
}

// One block of 256 threads per row, any length: two passes over the row.
__global__ void __launch_bounds__(256)
k_i8_quant_rows(const uint16_t* __restrict__ x, int64_t m, int64_t k, int8_t* __restrict__ x8, float* __restrict__ scale) {
  __shared__ uint32_t red[4];
  for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
    const uint16_t* xr = x + row * k;
    int8_t* qr = x8 + row * k;
    uint32_t mx = 0;
    for (int64_t i = threadIdx.x; i < k; i += 256) mx = amax_bits(mx, xr[i]);
    mx = wave_max(mx);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mx;
    __syncthreads();
    mx = max(max(red[0], red[1]), max(red[2], red[3]));
    __syncthreads();
    const float amax = __uint_as_float(mx);
    const bool finite = mx < 0x7F800000u, zero = mx == 0;
    const Coder c = coder_of(amax);
    if (threadIdx.x == 0) scale[row] = finite ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7FC00000u);
    for (int64_t i = threadIdx.x; i < k; i += 256)
      qr[i] = finite && !zero ? (int8_t)c.code(bf16_to_f32(xr[i])) : (int8_t)0;
  }
}

}  // namespace

hipError_t launch_i8_quant_rows(const uint16_t* x, int64_t m, int64_t k, int8_t* x8, float* s, hipStream_t st) {
  const int64_t blocks = m < 65536 ? m : 65536;
  hipLaunchKernelGGL(k_i8_quant_rows, dim3((unsigned)blocks), dim3(256), 0, st, x, m, k, x8, s);
  return hipGetLastError();
}

namespace {

// bf16(scale * code): one rounding of the fp32 product, 16 codes a thread.
__global__ void __launch_bounds__(256)
k_i8_dequant_rows(const int8_t* __restrict__ q, const float* __restrict__ s, int64_t rows, int64_t kc,
                  uint16_t* __restrict__ out) {
  const int64_t n = rows * kc;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const float sc = s[i / kc];
    const u32x4_t v = ld16(q + 16 * i);
    st16(out + 16 * i, i8x8_bf16_scaled(v[0], v[1], sc));
    st16(out + 16 * i + 8, i8x8_bf16_scaled(v[2], v[3], sc));
  }
}

// Rows of n values into rows of np, zeros behind: eight values a thread.
__global__ void __launch_bounds__(256)
k_i8_pad_rows(const uint16_t* __restrict__ x, int64_t rows, int64_t n, int64_t nc, uint16_t* __restrict__ out) {
  const int64_t total = rows * nc;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / nc, c = (i - row * nc) * 8;
    const uint16_t* xr = x + row * n;
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = c + 2 * j < n ? xr[c + 2 * j] : 0u, hi = c + 2 * j + 1 < n ? xr[c + 2 * j + 1] : 0u;
      v[j] = lo | (hi << 16);
    }
    st16(out + 8 * i, v);
  }
}

unsigned blocks_for(int64_t threads) {
  const int64_t b = (threads + 255) / 256;
  return (unsigned)(b < 16384 ? b : 16384);
}

}  // namespace

hipError_t launch_i8_dequant_rows(const int8_t* q, const float* s, int64_t rows, int64_t k, uint16_t* out, hipStream_t st) {
  const int64_t kc = k / 16;
  hipLaunchKernelGGL(k_i8_dequant_rows, dim3(blocks_for(rows * kc)), dim3(256), 0, st, q, s, rows, kc, out);
  return hipGetLastError();
}

hipError_t launch_i8_pad_rows(const uint16_t* x, int64_t rows, int64_t n, int64_t np, uint16_t* out, hipStream_t st) {
  hipLaunchKernelGGL(k_i8_pad_rows, dim3(blocks_for(rows * (np / 8))), dim3(256), 0, st, x, rows, n, np / 8, out);
  return hipGetLastError();
}

}  // namespace hm
