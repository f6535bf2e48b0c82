// Rows of the 8-bit integer layers: quantization per token (the codes that the
// product multiplies, and what a training step keeps of its activations), the
// copies that the gradients need (bf16 forms of 8-bit rows, padded odd rows).
#include <hip/hip_runtime.h>

#include "common.h"
#include "i8.h"
#include "i8_tile.h"

namespace hm {

namespace {

// The code of x in a row with largest magnitude amax is the whole number
// nearest to v = 127 x / amax, ties to even.  v is a ratio of whole numbers:
// with 8-bit significands X and A, v = 127 X / (A 2^c), c >= 0, and v - (j + 1/2) =
// (254 X - (2j + 1) A 2^c) / (2 A 2^c).  For a tie that v does not meet the numerator is a whole number
// other than 0, so the distance is at least 1 / (2 A 2^c) = v / (254 X) > v 2^-16.  The fp32
// product x (127 / amax) has two roundings, at most 2^-23 of v.  So rounding it to 19
// significant bits (the integer add and mask; it moves a value by at most 2^-19
// of itself) brings every tie to its exact value and moves nothing else across
// one; the second rounding, to whole numbers, then sees what the ratio itself
// would give.
// The rounding itself is the addition of 1.5 x 2^23, which leaves the code in the
// low byte of the sum.
struct Coder {
  float inv;                 // 127 / (amax pre), 0 for a row without codes
  float pre;                 // a power of two that keeps 127 / (amax pre) and the products in range
  __device__ __forceinline__ uint32_t code(float x) const {          // in the low byte
    const float t = (x * pre) * inv;
    return __float_as_uint(__uint_as_float((__float_as_uint(t) + 16u) & ~31u) + 12582912.0f);
  }
};

// A row's coder and scale from the bits of its largest magnitude.
__device__ __forceinline__ Coder coder_of(uint32_t bits, float& scale) {
  const float amax = __uint_as_float(bits);
  const bool finite = bits < 0x7F800000u;
  scale = finite ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7FC00000u);
  // by 2^100 for tiny rows (exact), by 2^-30 for huge ones (exact for every value whose code is not 0)
  Coder c;
  c.pre = amax < 0x1p-100f ? 0x1p100f : (amax > 0x1p100f ? 0x1p-30f : 1.0f);
  c.inv = finite && bits ? __fdiv_rn(127.0f, amax * c.pre) : 0.0f;
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

// Codes of eight values; a row with an infinity or NaN has none (0).
__device__ __forceinline__ u32x2_t codes8(u32x4_t v, const Coder& c, bool none) {
  u32x2_t r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = c.code(lo_bf16(v[2 * h])), b = c.code(hi_bf16(v[2 * h]));
    const uint32_t d = c.code(lo_bf16(v[2 * h + 1])), e = c.code(hi_bf16(v[2 * h + 1]));
    // low bytes of the four: selectors 4..7 name bytes of the first operand, 0..3 of the second
    const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), de = __builtin_amdgcn_perm(e, d, 0x0c0c0400u);
    r[h] = none ? 0u : ab | (de << 16);
  }
  return r;
}

typedef uint32_t u32x2_a1_t __attribute__((ext_vector_type(2), aligned(1)));
// Eight codes of a row of any length at any byte address.
__device__ __forceinline__ void put8(int8_t* row, int64_t k, int64_t at, u32x2_t v) {
  if (at + 7 < k) {
    *reinterpret_cast<u32x2_a1_t*>(row + at) = v;
  } else {
    for (int e = 0; at + e < k; ++e) row[at + e] = (int8_t)(v[e >> 2] >> (8 * (e & 3)));
  }
}

// Rows of up to 512 W CH values: W waves a row (four waves a block), lane L
// keeping the row's 16-byte chunks c 64 W + L in registers, so that the row is
// read once and all of its loads are in flight together.  Rows need no alignment.
template <int CH, int W>
__global__ void __launch_bounds__(256)
k_i8_quant_rows(const uint16_t* __restrict__ x, int64_t m, int64_t k, int8_t* __restrict__ x8, float* __restrict__ scale) {
  __shared__ uint32_t red[4];
  const int lane = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  for (int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x; row < m;
       row += (int64_t)gridDim.x * (4 / W)) {
    const uint16_t* xr = x + row * k;
    u32x4_t v[CH];
    uint32_t mx = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) v[c] = load8(xr, k, 8 * ((int64_t)c * 64 * W + lane));
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) mx = amax_bits(mx, v[c][j]);
    mx = wave_max(mx);
    if (W > 1) {
      if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mx;
      __syncthreads();
      mx = max(max(red[0], red[1]), max(red[2], red[3]));
      __syncthreads();
    }
    float s;
    const Coder co = coder_of(mx, s);
    if (lane == 0) scale[row] = s;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t at = 8 * ((int64_t)c * 64 * W + lane);
      if (at < k) put8(x8 + row * k, k, at, codes8(v[c], co, mx >= 0x7F800000u));
    }
  }
}

// Longer rows: a block each, two passes over the row.
__global__ void __launch_bounds__(256)
k_i8_quant_long_rows(const uint16_t* __restrict__ x, int64_t m, int64_t k, int8_t* __restrict__ x8, float* __restrict__ scale) {
  __shared__ uint32_t red[4];
  for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
    const uint16_t* xr = x + row * k;
    uint32_t mx = 0;
    for (int64_t i = threadIdx.x * 8; i < k; i += 256 * 8) {
      const u32x4_t v = load8(xr, k, i);
#pragma unroll
      for (int j = 0; j < 4; ++j) mx = amax_bits(mx, v[j]);
    }
    mx = wave_max(mx);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mx;
    __syncthreads();
    mx = max(max(red[0], red[1]), max(red[2], red[3]));
    __syncthreads();
    float s;
    const Coder co = coder_of(mx, s);
    if (threadIdx.x == 0) scale[row] = s;
    for (int64_t i = threadIdx.x * 8; i < k; i += 256 * 8)
      put8(x8 + row * k, k, i, codes8(load8(xr, k, i), co, mx >= 0x7F800000u));
  }
}

template <int CH, int W>
void go(const uint16_t* x, int64_t m, int64_t k, int8_t* x8, float* s, hipStream_t st) {
  const int64_t want = (m * W + 3) / 4;
  hipLaunchKernelGGL((k_i8_quant_rows<CH, W>), dim3((unsigned)(want < 65536 ? want : 65536)), dim3(256), 0, st, x, m, k, x8, s);
}

}  // namespace

// A wave a row up to 2048 values, a block above.
hipError_t launch_i8_quant_rows(const uint16_t* x, int64_t m, int64_t k, int8_t* x8, float* s, hipStream_t st) {
  if (k <= 512) go<1, 1>(x, m, k, x8, s, st);
  else if (k <= 1024) go<2, 1>(x, m, k, x8, s, st);
  else if (k <= 2048) go<4, 1>(x, m, k, x8, s, st);
  else if (k <= 4096) go<2, 4>(x, m, k, x8, s, st);
  else if (k <= 8192) go<4, 4>(x, m, k, x8, s, st);
  else if (k <= 16384) go<8, 4>(x, m, k, x8, s, st);
  else hipLaunchKernelGGL(k_i8_quant_long_rows, dim3((unsigned)(m < 65536 ? m : 65536)), dim3(256), 0, st, x, m, k, x8, s);
  return hipGetLastError();
}

namespace {

// The copies that a gradient needs, in one launch.  Codes: bf16(scale * code), one
// rounding of the fp32 product (a factor of the bf16 MFMA, see Codes), 16 a thread.  Rows of n values into rows of 8 nc, zeros behind: eight a thread.
__global__ void __launch_bounds__(256)
k_i8_copies(I8Copies c) {
  const int64_t n0 = c.rows[0] * c.kc, n1 = n0 + c.rows[1] * c.kc, total = n1 + c.m * c.nc;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    if (i < n1) {
      const int w = i >= n0;
      const int64_t at = w ? i - n0 : i;
      const float sc = (w ? c.s[1] : c.s[0])[at / c.kc];
      const u32x4_t v = ld16((w ? c.q[1] : c.q[0]) + 16 * at);
      uint16_t* out = (w ? c.out[1] : c.out[0]) + 16 * at;
      st16(out, i8x8_bf16_scaled(v[0], v[1], sc));
      st16(out + 8, i8x8_bf16_scaled(v[2], v[3], sc));
    } else {
      const int64_t at = i - n1, row = at / c.nc, col = (at - row * c.nc) * 8;
      const uint16_t* xr = c.dy + row * c.n;
      u32x4_t v;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = col + 2 * j < c.n ? xr[col + 2 * j] : 0u, hi = col + 2 * j + 1 < c.n ? xr[col + 2 * j + 1] : 0u;
        v[j] = lo | (hi << 16);
      }
      st16(c.pad + 8 * at, v);
    }
  }
}

unsigned blocks_for(int64_t threads) {
  const int64_t b = (threads + 255) / 256;
  return (unsigned)(b < 16384 ? b : 16384);
}

}  // namespace

hipError_t launch_i8_copies(const I8Copies& c, hipStream_t st) {
  const int64_t threads = (c.rows[0] + c.rows[1]) * c.kc + c.m * c.nc;
  if (!threads) return hipSuccess;
  hipLaunchKernelGGL(k_i8_copies, dim3(blocks_for(threads)), dim3(256), 0, st, c);
  return hipGetLastError();
}

}  // namespace hm
