// dx of the 8-bit integer layers for few rows: dx[q][p] = sum_n dy[q][n] bf16(s[n] w8[n][p]).
//
// As the products for few rows: a block has 64 columns p against a group of 32 QB rows
// of dy, and its W waves split the contraction, each by itself: steps w, w + W, ... of
// 64 rows n of the weights (64 bytes of each) and of 128 bytes of every row of dy, through
// LDS by direct copies, no barrier before the sums meet.  The codes are read transposed
// (a lane then has eight n of one column), turned into bf16 with the scale of their row
// and multiplied on 32x32x16 MFMAs.  The waves' fp32 sums are added in order.
//
// Two waves a SIMD: one alone issues a VALU instruction every eight clocks, two every four
// (32 rows, m = 102, n = 11221, k = 1536: eight waves 31.3 us, four 35.7).  A step's copies are on
// their way while it is multiplied, and those of the other waves; more steps ahead bring nothing (36.3 with
// three).  Against the 128 x 128 tiles, whose parts need a second launch: m = 333, n = 7168, k = 2048 23.4 us for 30.4,
// m = 851, n = 3968, k = 1792 25.6 for 32.2, m = 70, n = 3802, k = 4096 13.9 for 21.6.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "common.h"
#include "i8.h"
#include "i8_tile.h"

namespace hm {

namespace {

constexpr int kCodes = 4096;                       // 64 rows x 64 bytes
constexpr int kScaleBytes = 256;

// LDS of a wave: a step, then its sums.  QB: 32-row blocks of dy
template <int QB> constexpr int kDxOwn = kCodes + QB * 4096 + kScaleBytes > QB * 8192 ? kCodes + QB * 4096 + kScaleBytes : QB * 8192;

template <int QB, int W>
__global__ void __launch_bounds__(64 * W)
k_i8_few_dx(TileArgs a, uint32_t total, int groups) {
  extern __shared__ __align__(1024) uint8_t lds[];
  constexpr int kStep = kCodes + QB * 4096, kOwn = kDxOwn<QB>;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the groups of rows after each other on an XCD, whose L2 then has the weights
  const uint32_t t0 = number_of(total, blockIdx.x, gridDim.x, 0);
  if (t0 >= total) return;
  const uint32_t tc = t0 / (uint32_t)groups;
  const int64_t c0 = (int64_t)tc * 64, r0 = (int64_t)(t0 - tc * groups) * (32 * QB);
  const int rows = (int)min((int64_t)(32 * QB), a.rows - r0);
  uint8_t* const own = lds + wave * kOwn;
  const int all = (int)((a.kbytes + 127) / 128);   // steps of all waves
  const uint32_t ldp = (uint32_t)a.p_ld, ldq = (uint32_t)a.q_ld;
  const uint8_t* pp = a.p + c0 + (int64_t)wave * 64 * ldp;
  const uint8_t* pq = a.q + r0 * ldq + wave * 128;
  int64_t lp = a.p_bytes - c0 - (int64_t)wave * 64 * ldp, lq = (int64_t)rows * ldq - wave * 128;
  const rsrc_t rs = make_rsrc(a.ps, (uint64_t)a.terms * 4);
  uint32_t sv = wave * 256 + lane * 4;
  // copy i of codes: rows 16 i + lane / 4, 16-byte chunk c at place c ^ 2 ((row >> 2) & 1): the eight rows and 32
  // bytes that two groups of lanes read together then lie in different banks
  const uint32_t vp = (uint32_t)(lane >> 2) * ldp + 16 * ((lane & 3) ^ (2 * ((lane >> 4) & 1)));
  // copy i of dy: rows 8 i + lane / 8, chunk c at place c ^ ((row >> 1) & 7)
  const int in = (int)(a.kbytes & 127);
  uint32_t vq[2];
  uint32_t tail = 0;                               // bit i: the lane's chunk lies behind the contraction in the last step
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int chunk = (lane & 7) ^ ((lane >> 4) | (4 * i));
    vq[i] = (uint32_t)(8 * i + (lane >> 3)) * ldq + 16 * chunk;
    if (in && 16 * chunk >= in) tail |= 1u << i;
  }
  int next = wave;                                 // step to copy
  auto fetch = [&]() __attribute__((always_inline)) {
    const bool any = next < all;                   // past the end: zeros
    const rsrc_t rp = make_rsrc(pp, any && lp > 0 ? (uint64_t)lp : 0), rq = make_rsrc(pq, any ? (uint64_t)lq : 0);
    const uint32_t cut = next == all - 1 ? tail : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) b2lds16(rp, vp + (uint32_t)i * 16 * ldp, 0u, own + i * 1024);
#pragma unroll
    for (int i = 0; i < 4 * QB; ++i)
      b2lds16(rq, (vq[i & 1] + (uint32_t)(i >> 1) * 16 * ldq) | ((cut >> (i & 1)) & 1u ? 0xFFFFFFFFu : 0u), 0u, own + kCodes + i * 1024);
    b2lds4(rs, sv, 0u, own + kStep);
    pp += (int64_t)64 * W * ldp;
    lp -= (int64_t)64 * W * ldp;
    pq += 128 * W;
    lq -= 128 * W;
    sv += 256 * W;
    next += W;
  };
  fetch();
  // codes: lane l of group g supplies row 8 (g >> 1) + l / 2, eight of the 16 bytes of chunk g & 1 (block b: 2 b + (g & 1)), and gets
  // column l of the eight rows
  const uint32_t base = (uint32_t)(uintptr_t)(lds_void_t*)own;
  const int g = lane >> 4, l = lane & 15, l32 = lane & 31, hi = lane >> 5;
  uint32_t ap[2], aq[4];
#pragma unroll
  for (int b = 0; b < 2; ++b) ap[b] = base + (8 * (g >> 1) + (l >> 1)) * 64 + 16 * ((2 * b + (g & 1)) ^ (2 * ((l >> 3) & 1))) + 8 * (l & 1);
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) aq[ks] = base + kCodes + l32 * 128 + 16 * ((2 * ks + hi) ^ ((l32 >> 1) & 7));
  const uint32_t as = base + kStep + 32 * (g >> 1);

  f32x16_t acc[2][QB];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < QB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  typedef __attribute__((address_space(3))) f32x4_t lds_f32x4_t;
  for (int steps = (all - wave + W - 1) / W; steps > 0; --steps) {
    __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
    u32x2_t p[2][4];
    u32x4_t q[QB][4];
    f32x4_t s[4][2];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
      for (int b = 0; b < 2; ++b) p[b][ks] = read_tr8((const lds_i32x2_t*)(ap[b] + ks * 16 * 64));
#pragma unroll
      for (int h = 0; h < 2; ++h) s[ks][h] = *(const lds_f32x4_t*)(as + ks * 64 + h * 16);
#pragma unroll
      for (int b = 0; b < QB; ++b) q[b][ks] = *(const lds_u32x4_t*)(aq[ks] + b * 4096);
    }
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");             // the step is in registers
    __builtin_amdgcn_sched_barrier(0);
    fetch();
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const u32x2_t x = Codes::values(p[b][ks][0], s[ks][0]), y = Codes::values(p[b][ks][1], s[ks][1]);
#pragma unroll
        for (int j = 0; j < QB; ++j) acc[b][j] = Mma<uint16_t>::run((u32x4_t){x[0], x[1], y[0], y[1]}, q[j][ks], acc[b][j]);
      }
  }
  // the wave's sums take the place of its steps
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  auto sums = [&](int w, int i, int j, int x) -> f32x4_t& { return reinterpret_cast<f32x4_t*>(lds + w * kOwn)[((i * QB + j) * 4 + x) * 64 + lane]; };
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < QB; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x) sums(wave, i, j, x) = (f32x4_t){acc[i][j][4 * x], acc[i][j][4 * x + 1], acc[i][j][4 * x + 2], acc[i][j][4 * x + 3]};
  __syncthreads();
  // half a 32 x 32 block at a time: 16 columns, eight a lane
  for (int n = wave; n < 4 * QB; n += W) {
    const int i = n & 1, x = (n >> 1) & 1, u = n >> 2;
    u32x2_t o[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      f32x4_t v = sums(0, i, u, 2 * x + y);
#pragma unroll
      for (int w = 1; w < W; ++w) v += sums(w, i, u, 2 * x + y);
      o[y] = (u32x2_t){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
    const u32x4_t v = eight(o[0], o[1]);
    const int r = u * 32 + l32;
    if (r < rows) st16(a.out + (r0 + r) * a.cols + c0 + i * 32 + 16 * x + 8 * hi, v);
  }
}

template <int QB, int W>
hipError_t go(const TileArgs& a, hipStream_t st) {
  constexpr int kLds = W * kDxOwn<QB>;
  auto kern = &k_i8_few_dx<QB, W>;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (attr != hipSuccess) return attr;
  const int groups = (int)((a.rows + 32 * QB - 1) / (32 * QB));
  const uint32_t total = (uint32_t)(a.cols / 64 * groups);
  hipLaunchKernelGGL(kern, dim3(8 * ((total + 7) / 8)), dim3(64 * W), kLds, st, a, total, groups);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_few_dx(const TileArgs& a, int rows, hipStream_t st) {
  switch (rows) {
    case 32: return go<1, 8>(a, st);
    case 64: return go<2, 8>(a, st);
    default: return go<4, 4>(a, st);
  }
}

}  // namespace hm
