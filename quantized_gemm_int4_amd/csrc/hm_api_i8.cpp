// C ABI entry points of the 8-bit integer layers: argument checks, workspace
// layout and launches.  Every check runs before any launch; nothing is
// allocated.
#include <hip/hip_runtime.h>
#include <stdio.h>

#include <algorithm>
#include <initializer_list>

#include "../../include/hm.h"
#include "common.h"
#include "i8.h"

#define HM_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace hm;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// An array of a call.  No array is longer than the card's memory (288 GB), so
// lengths end at 2^39 and ends do not wrap.
struct Span {
  const void* p;             // null, or no bytes: no array
  uint64_t bytes;
};
bool meets(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  constexpr uint64_t kMost = 1ull << 39;
  const uint64_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + std::min(b.bytes, kMost) && y < x + std::min(a.bytes, kMost);
}
// Whether an output or the workspace meets an input or another of them.
bool overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (meets(*o, i)) return true;
    for (const Span* p = o + 1; p != outs.end(); ++p)
      if (meets(*o, *p)) return true;
  }
  return false;
}

constexpr int64_t kMaxRows = 8388480;         // 65535 x 128, as hm_gemm
constexpr int64_t kMaxCols = 1ll << 22;       // 256 rows of bf16 gradients stay under 2^31 bytes
constexpr int64_t kMaxK = 130944;             // below 2^31 / 128^2: no sum of products of two int8 leaves the int32 range
constexpr int64_t kMaxTiles = 1ll << 23;      // of 320 threads each: a launch has less than 2^32

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool tiles_fit(int64_t rows, int64_t cols) { return div_up(rows, kI8Tile) * div_up(cols, kI8Tile) <= kMaxTiles; }

// n: rows of the weights (gated: 2 d)
hm_status check_sizes(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || m > kMaxRows || n < 1 || n > kMaxCols || k < 128 || (k % 128) != 0 || k > kMaxK) return HM_ERR_SHAPE;
  return tiles_fit(m, n) ? HM_OK : HM_ERR_SHAPE;
}

hm_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!need) return HM_OK;
  if (!ws) return HM_ERR_NULL;
  if (ws_bytes < need) return HM_ERR_WORKSPACE;
  return aligned(ws, 256) ? HM_OK : HM_ERR_ALIGN;
}

hm_status done(hipError_t e) { return e == hipSuccess ? HM_OK : HM_ERR_HIP; }

TileArgs product(const int8_t* x8, const float* xs, const int8_t* w8, const float* ws, int64_t m, int64_t n, int64_t k,
                 uint16_t* out) {
  TileArgs a{};
  a.p = (const uint8_t*)w8;
  a.p_ld = k;
  a.p_bytes = n * k;
  a.q = (const uint8_t*)x8;
  a.q_ld = k;
  a.q_bytes = m * k;
  a.rows = m;
  a.cols = n;
  a.kbytes = k;
  a.ps = ws;
  a.qs = xs;
  a.out = out;
  return a;
}

// How a product runs: which tiles, and how the last ones are cut.
struct Plan {
  bool few, big;
  FewPlan fewer;
  int few_dx;                // rows of a group of the kernel for few rows of a gradient, 0: tiles
  TilePlan tiles;
  size_t part;               // workspace bytes of the cut tiles' sums
  int64_t ns;                // estimate of the time
};

// Nanoseconds of up to 256 tiles at once, one a compute unit, by the contraction's steps
// of 128 bytes, taken in twos: estimates fitted to measured calls, which choose between kernels that all give the
// same results (gradients: up to the order of their sums).  Of 400 choices at 80 drawn sizes (m 1 to 8192, n 64 to
// 14336, k 256 to 7168; product, gated block, its gradient, dx, dw) half took within 1.5 % of the fastest of all kernels
// forced in turn, nine of ten within 10 %, the worst 1.3 times it, but for one of a call of 4 us (1.6).
// Copies from L2 bound the small tiles, the conversion those that turn codes into bf16, copies
// and the matrix cores the large ones.
constexpr int kCus = 256;
enum Operands { INT8, INT8_GRAD, CODES, COPY };    // int8 products, the gated gradient; gradients with P as codes, as a bf16 copy
int64_t small_round(Operands o, int64_t tiles, int64_t steps) {
  return (steps + 1) / 2 * 2 * ((o == CODES ? 590 : 440) + 70 * tiles / kCus) + (o == INT8_GRAD ? 3400 : 2000) + 1700 * tiles / kCus;
}
// Two blocks a compute unit, up to 512 tiles at once: the start and the end of one go with the other's steps, but each
// has only half of the copies on their way.
int64_t two_round(Operands o, int64_t tiles, int64_t steps) {
  const int64_t one = std::min<int64_t>(tiles, kCus), more = tiles - one, grad = o == INT8_GRAD;
  const int64_t step = o == CODES ? (more ? 930 + 170 * more / kCus : 600 + 160 * one / kCus)
                                  : (more ? 830 + 150 * more / kCus : 500 + 130 * one / kCus);
  return (steps + 1) / 2 * 2 * step + 1700 + 1400 * grad + (1700 * one + (200 + 1600 * grad) * more) / kCus;
}
int64_t big_round(Operands o, int64_t tiles, int64_t steps) {
  return (steps + 1) / 2 * 2 * (1100 + 430 * tiles / kCus) + (o == INT8_GRAD ? 16000 : 9500);
}
// Few rows: nanoseconds of the blocks one compute unit has, as many at a time as LDS takes.  A block reads
// its weights at 40 bytes a nanosecond and its rows of x, which others have brought into L2, at 100,
// and all of them no faster than the memory gives the weights (k = 4096, m = 64, n = 14336: four blocks of 16
// weight rows a block 17.8 us, two 20.2, one 26.6; k = 5248, m = 48, n = 3985: one 9.5, two 11.1).
int64_t memory_time(int64_t cols, bool pairs, int64_t k) { return cols * (pairs ? 2 : 1) * k / 4900; }
int64_t few_time(int64_t rows, int64_t cols, bool pairs, int64_t k, FewPlan& p) {
  const int64_t blocks = div_up(rows, 16), least = div_up(blocks, 8), memory = memory_time(cols, pairs, k);
  int64_t best = 0;
  for (int64_t g = least; g <= 4 * least && g <= blocks; g *= 2) {
    const int64_t mb = div_up(blocks, g), groups = div_up(blocks, mb), rb = std::min(16 * mb, rows);
    for (int64_t nb = pairs ? 2 : 1; nb <= i8_few_most((int)mb, pairs); nb += pairs ? 2 : 1) {
      const int64_t rounds = div_up(div_up(cols, 16 * (pairs ? nb / 2 : nb)) * groups, kCus);
      const int64_t at_once = std::max<int64_t>(1, 160 / std::max(8 * (nb + mb), 4 * nb * mb));
      const int64_t base = div_up(rounds, at_once) * (3300 + 200 * nb + 80 * nb * mb);
      const int64_t t = std::max(rounds * (k * (nb * 40 + rb) / 100), memory) + base;
      if (!best || t < best) {
        best = t;
        p = {(int)groups, (int)(16 * mb), (int)nb};
      }
    }
  }
  return best;
}

// kbytes: of the contraction, as the operands' rows hold it.
Plan plan_tiles(int64_t rows, int64_t cols, bool pairs, int64_t kbytes, Operands o) {
  const int64_t steps = div_up(kbytes, 128);
  Plan p{};
  p.tiles.tiles_p = (int)div_up(cols, pairs ? kI8Tile / 2 : kI8Tile);
  p.tiles.tiles_q = (int)div_up(rows, kI8Tile);
  p.tiles.codes = o == CODES;
  const int64_t tiles = (int64_t)p.tiles.tiles_p * p.tiles.tiles_q, rest = tiles % kCus;
  int64_t best = rest ? small_round(o, rest, steps) : 0, cut = 1;
  for (int64_t c = 2; c <= 32 && rest && rest * c <= 2 * kCus && steps >= 4 * c; ++c) {
    // a second launch, and the sums written and read again
    const int64_t t = div_up(rest * c, kCus) * small_round(o, std::min<int64_t>(rest * c, kCus), div_up(steps, c)) + 4000 +
                      30 * rest * c;
    if (t < best) {
      best = t;
      cut = c;
    }
  }
  p.tiles.per = (int)std::max<int64_t>(1, div_up(steps, cut));
  p.tiles.cut = (int)std::max<int64_t>(1, div_up(steps, p.tiles.per));
  p.tiles.full = (int)(p.tiles.cut > 1 ? tiles - rest : tiles);
  p.part = p.tiles.cut > 1 ? (size_t)rest * p.tiles.cut * kI8Tile * kI8Tile * 4 : 0;
  p.ns = best + tiles / kCus * small_round(o, kCus, steps);
  const int64_t last = tiles % (2 * kCus);
  const int64_t two = tiles / (2 * kCus) * two_round(o, 2 * kCus, steps) + (last ? two_round(o, last, steps) : 0);
  if (two < p.ns) {
    p.tiles.two = 1;
    p.tiles.full = (int)tiles;
    p.tiles.cut = 1;
    p.tiles.per = (int)std::max<int64_t>(1, steps);
    p.part = 0;
    p.ns = two;
  }
  if (o == CODES) return p;                        // the large tiles take no codes
  const int64_t bigs = div_up(cols, pairs ? kI8Big / 2 : kI8Big) * div_up(rows, kI8Big);
  const int64_t t = bigs / kCus * big_round(o, kCus, steps) + (bigs % kCus ? big_round(o, bigs % kCus, steps) : 0);
  if (t < p.ns) {
    p.big = true;
    p.ns = t;
    p.part = 0;
  }
  return p;
}

// An int8 product.
Plan plan_product(int64_t rows, int64_t cols, bool pairs, int64_t k, Operands o = INT8) {
  Plan p = plan_tiles(rows, cols, pairs, k, o);
  // (2300: a launch, which few_time counts and the tiles' estimates do not)
  if (rows <= kI8Few && few_time(rows, cols, pairs, k, p.fewer) < std::max(p.ns, memory_time(cols, pairs, k) + 3000) + 2300) {
    p.few = true;
    p.part = 0;
  }
  return p;
}

// dx of few rows: groups of 32, 64 or 128 rows, of which a compute unit takes steps of 64 of the contraction in so
// many nanoseconds.
int64_t few_dx_time(int64_t rows, int64_t cols, int64_t kbytes, int& group) {
  int64_t best = 0;
  for (int r = 32; r <= 128; r *= 2) {
    const int64_t n = cols / 64 * div_up(rows, r), c = r == 32 ? 155 : r == 64 ? 190 : 260 + 160 * std::min<int64_t>(n, kCus) / kCus;
    const int64_t t = div_up(n, kCus) * (div_up(kbytes, 128) * c + (r == 32 ? 1000 : 3000)) + 3500;
    if (!best || t < best) {
      best = t;
      group = r;
    }
  }
  return best;
}

// One of the gradients: `terms` rows of the int8 operand, [terms][cols].
Plan plan_gradient(int64_t rows, int64_t cols, int64_t kbytes, int64_t terms) {
  const Plan codes = plan_tiles(rows, cols, false, kbytes, CODES);
  Plan copy = plan_tiles(rows, cols, false, kbytes, COPY);
  copy.ns += 3000 + terms * cols * 3 / 6000;       // making the copy: 6 TB/s
  return codes.ns < copy.ns ? codes : copy;
}

hipError_t multiply(const TileArgs& a, const Plan& p, int kind, void* part, hipStream_t st) {
  if (p.few) return launch_i8_few(a, p.fewer, kind, st);
  if (p.few_dx) return launch_i8_few_dx(a, p.few_dx, st);
  if (p.big) return launch_i8_big(a, kind, st);
  TilePlan t = p.tiles;
  t.part = part;
  return launch_i8_tile(a, t, kind, st);
}

// Byte offsets in the workspace of the gradient.
struct GradPlan {
  size_t dyp, w, x, part, total;
  int64_t np;                // columns of the padded copy of dy, 0: dy itself
  Plan dx, dw;
};
GradPlan plan_grad(int64_t m, int64_t n, int64_t k) {
  GradPlan g{};
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t o = at;
    at = align256(at + bytes);
    return o;
  };
  g.np = (n % 8) ? (n + 7) / 8 * 8 : 0;
  g.dw = plan_gradient(n, k, 2 * m, m);
  if (m == 0) return g;
  g.dx = plan_gradient(m, k, 2 * (g.np ? g.np : n), n);
  int group = 0;
  if (m <= 2 * kI8Few && few_dx_time(m, k, 2 * n, group) < g.dx.ns + 2300) {
    g.dx.few_dx = group;
    g.dx.tiles.codes = 1;
    g.dx.part = 0;
  }
  g.dyp = take((size_t)m * (size_t)g.np * 2);
  g.w = take(!g.dx.tiles.codes ? (size_t)n * (size_t)k * 2 : 0);
  g.x = take(!g.dw.tiles.codes ? (size_t)m * (size_t)k * 2 : 0);
  g.part = take(std::max(g.dx.part, g.dw.part));
  g.total = at;
  return g;
}

}  // namespace

HM_API hm_status hm_quant_int8_rows(const uint16_t* x, int64_t m, int64_t k, int8_t* x8, float* row_scale,
                                    hipStream_t stream) {
  if (m < 0 || k < 1) return HM_ERR_SHAPE;
  if (m == 0) return HM_OK;
  if (!x || !x8 || !row_scale) return HM_ERR_NULL;
  if (!aligned(x, 16) || !aligned(x8, 16) || !aligned(row_scale, 4)) return HM_ERR_ALIGN;
  if (k > (1ll << 39) / m) return HM_ERR_SHAPE;
  const uint64_t e = (uint64_t)m * (uint64_t)k;
  if (overlap({{x8, e}, {row_scale, 4ull * m}}, {{x, 2 * e}})) return HM_ERR_UNSUPPORTED;
  return done(launch_i8_quant_rows(x, m, k, x8, row_scale, stream));
}

// ------------------------------------------------------------------ products

HM_API hm_status hm_gemm_int8_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  if (hm_status s = check_sizes(m, n, k)) return s;
  if (!bytes) return HM_ERR_NULL;
  *bytes = m ? plan_product(m, n, false, k).part : 0;
  return HM_OK;
}

HM_API hm_status hm_gemm_int8(const int8_t* x8, const float* x_scales, const int8_t* w8, const float* w_scales,
                              int64_t m, int64_t n, int64_t k, uint16_t* y, void* ws, size_t ws_bytes,
                              hipStream_t stream) {
  if (hm_status s = check_sizes(m, n, k)) return s;
  if (m == 0) return HM_OK;
  if (!x8 || !x_scales || !w8 || !w_scales || !y) return HM_ERR_NULL;
  if (!aligned(x8, 16) || !aligned(w8, 16) || !aligned(y, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4))
    return HM_ERR_ALIGN;
  const Plan p = plan_product(m, n, false, k);
  const size_t need = p.part;
  if (hm_status s = check_ws(ws, ws_bytes, need)) return s;
  const uint64_t um = m, un = n, uk = k;
  if (overlap({{y, 2 * um * un}, {ws, need}}, {{x8, um * uk}, {x_scales, 4 * um}, {w8, un * uk}, {w_scales, 4 * un}}))
    return HM_ERR_UNSUPPORTED;
  return done(multiply(product(x8, x_scales, w8, w_scales, m, n, k, y), p, I8_FORWARD, ws, stream));
}

// ---------------------------------------------------------------- gated block

namespace {

hm_status check_gated(int64_t m, int64_t n, int64_t k) {
  if (hm_status s = check_sizes(m, n, k)) return s;
  return (n % 2) ? HM_ERR_SHAPE : HM_OK;
}

}  // namespace

HM_API hm_status hm_gemm_int8_gated_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  if (hm_status s = check_gated(m, n, k)) return s;
  if (!bytes) return HM_ERR_NULL;
  *bytes = m ? plan_product(m, n / 2, true, k).part : 0;
  return HM_OK;
}

HM_API hm_status hm_gemm_int8_gated(const int8_t* x8, const float* x_scales, const int8_t* w8, const float* w_scales,
                                    int64_t m, int64_t n, int64_t k, uint16_t* h, void* ws, size_t ws_bytes,
                                    hipStream_t stream) {
  if (hm_status s = check_gated(m, n, k)) return s;
  if (m == 0) return HM_OK;
  if (!x8 || !x_scales || !w8 || !w_scales || !h) return HM_ERR_NULL;
  if (!aligned(x8, 16) || !aligned(w8, 16) || !aligned(h, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4))
    return HM_ERR_ALIGN;
  const Plan p = plan_product(m, n / 2, true, k);
  const size_t need = p.part;
  if (hm_status s = check_ws(ws, ws_bytes, need)) return s;
  const uint64_t um = m, un = n, uk = k;
  if (overlap({{h, um * un}, {ws, need}}, {{x8, um * uk}, {x_scales, 4 * um}, {w8, un * uk}, {w_scales, 4 * un}}))
    return HM_ERR_UNSUPPORTED;
  TileArgs a = product(x8, x_scales, w8, w_scales, m, n, k, h);
  a.cols = n / 2;
  a.p_bytes = n / 2 * k;
  return done(multiply(a, p, I8_GATED, ws, stream));
}

HM_API hm_status hm_gemm_int8_gated_grad_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  if (hm_status s = check_gated(m, n, k)) return s;
  if (!bytes) return HM_ERR_NULL;
  *bytes = m ? plan_product(m, n / 2, true, k, INT8_GRAD).part : 0;
  return HM_OK;
}

HM_API hm_status hm_gemm_int8_gated_grad(const uint16_t* dh, const int8_t* x8, const float* x_scales, const int8_t* w8,
                                         const float* w_scales, int64_t m, int64_t n, int64_t k, uint16_t* dgu, void* ws,
                                         size_t ws_bytes, hipStream_t stream) {
  if (hm_status s = check_gated(m, n, k)) return s;
  if (m == 0) return HM_OK;
  if (!dh || !x8 || !x_scales || !w8 || !w_scales || !dgu) return HM_ERR_NULL;
  if (!aligned(dh, 16) || !aligned(x8, 16) || !aligned(w8, 16) || !aligned(dgu, 16) || !aligned(x_scales, 4) ||
      !aligned(w_scales, 4))
    return HM_ERR_ALIGN;
  const Plan p = plan_product(m, n / 2, true, k, INT8_GRAD);
  const size_t need = p.part;
  if (hm_status s = check_ws(ws, ws_bytes, need)) return s;
  const uint64_t um = m, un = n, uk = k;
  if (overlap({{dgu, 2 * um * un}, {ws, need}},
              {{dh, um * un}, {x8, um * uk}, {x_scales, 4 * um}, {w8, un * uk}, {w_scales, 4 * un}}))
    return HM_ERR_UNSUPPORTED;
  TileArgs a = product(x8, x_scales, w8, w_scales, m, n, k, dgu);
  a.cols = n / 2;
  a.p_bytes = n / 2 * k;
  a.dh = dh;
  return done(multiply(a, p, I8_GATED_GRAD, ws, stream));
}

// ------------------------------------------------------------------- gradient

namespace {

hm_status check_grad(int64_t m, int64_t n, int64_t k) {
  if (hm_status s = check_sizes(m, n, k)) return s;
  return tiles_fit(m, k) && tiles_fit(n, k) ? HM_OK : HM_ERR_SHAPE;
}

}  // namespace

HM_API hm_status hm_gemm_int8_grad_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  if (hm_status s = check_grad(m, n, k)) return s;
  if (!bytes) return HM_ERR_NULL;
  *bytes = plan_grad(m, n, k).total;
  return HM_OK;
}

HM_API hm_status hm_gemm_int8_grad(const uint16_t* dy, const int8_t* x8, const float* x_scales, const int8_t* w8,
                                   const float* w_scales, int64_t m, int64_t n, int64_t k, uint16_t* dx, uint16_t* dw,
                                   void* ws, size_t ws_bytes, hipStream_t stream) {
  if (hm_status s = check_grad(m, n, k)) return s;
  if (!dx && !dw) return HM_ERR_NULL;
  if (m == 0 && !dw) return HM_OK;
  if (!aligned(dx, 16) || !aligned(dw, 16)) return HM_ERR_ALIGN;
  TileArgs a{};
  if (m) {
    if (!dy || (dw && (!x8 || !x_scales)) || (dx && (!w8 || !w_scales))) return HM_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(x8, 16) || !aligned(w8, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4))
      return HM_ERR_ALIGN;
  }
  const GradPlan g = plan_grad(m, n, k);
  if (hm_status s = check_ws(ws, ws_bytes, g.total)) return s;
  const uint64_t um = m, un = n, uk = k;
  if (overlap({{dx, 2 * um * uk}, {dw, 2 * un * uk}, {ws, g.total}},
              {{dy, 2 * um * un}, {x8, um * uk}, {x_scales, 4 * um}, {w8, un * uk}, {w_scales, 4 * un}}))
    return HM_ERR_UNSUPPORTED;
  uint8_t* at = (uint8_t*)ws;
  // what the products read in place of the arguments, in one launch
  I8Copies c{};
  c.kc = k / 16;
  c.dy = dy;
  c.pad = (uint16_t*)(at + g.dyp);
  c.m = m;
  c.n = n;
  c.nc = g.np / 8;
  auto copy = [&](int i, const int8_t* q, const float* s, int64_t rows, size_t to) {
    c.q[i] = q;
    c.s[i] = s;
    c.rows[i] = rows;
    c.out[i] = (uint16_t*)(at + to);
  };
  if (dx && m && !g.dx.tiles.codes) copy(0, w8, w_scales, n, g.w);
  if (dw && !g.dw.tiles.codes) copy(1, x8, x_scales, m, g.x);
  hipError_t e = launch_i8_copies(c, stream);
  const int64_t ldy = g.np ? g.np : n;
  a.q = g.np && m ? (const uint8_t*)c.pad : (const uint8_t*)dy;
  a.q_ld = 2 * ldy;
  a.q_bytes = 2 * m * ldy;
  a.cols = k;
  // P: the int8 operand, as codes or as its bf16 copy
  auto side = [&](const Plan& p, const int8_t* q8, const float* scales, int64_t rows, size_t to) {
    const bool codes = p.tiles.codes;
    a.p = codes ? (const uint8_t*)q8 : at + to;
    a.p_ld = (codes ? 1 : 2) * k;
    a.p_bytes = rows * a.p_ld;
    a.ps = scales;
    a.terms = rows;
  };
  if (dx && m && e == hipSuccess) {
    side(g.dx, w8, w_scales, n, g.w);
    a.rows = m;
    a.kbytes = 2 * ldy;
    a.out = dx;
    e = multiply(a, g.dx, I8_DX, at + g.part, stream);
  }
  if (dw && e == hipSuccess) {
    side(g.dw, x8, x_scales, m, g.x);
    a.rows = n;
    a.kbytes = 2 * m;
    a.out = dw;
    e = multiply(a, g.dw, I8_DW, at + g.part, stream);
  }
  return done(e);
}

// ----------------------------------------------------------------------- plan

namespace {

int say(const Plan& p, bool pairs, int64_t rows, int64_t cols, char* buf, size_t len) {
  if (p.few)
    return snprintf(buf, len, "few rows: %d groups of %d row blocks, weight blocks %d", p.fewer.groups, p.fewer.rows / 16, p.fewer.nb);
  if (p.few_dx) return snprintf(buf, len, "few rows: groups of %d", p.few_dx);
  if (p.big) return snprintf(buf, len, "tiles 256x256: %lld", (long long)(div_up(rows, kI8Big) * div_up(cols, pairs ? kI8Big / 2 : kI8Big)));
  return snprintf(buf, len, "tiles 128x128%s%s: %d whole, %d in %d parts", p.tiles.codes ? " of codes" : "", p.tiles.two ? ", two at once" : "", p.tiles.full,
                  p.tiles.tiles_p * p.tiles.tiles_q - p.tiles.full, p.tiles.cut);
}

}  // namespace

HM_API hm_status hm_gemm_int8_plan(int32_t op, int64_t m, int64_t n, int64_t k, char* buf, size_t buf_len) {
  if (op < HM_INT8_GEMM || op > HM_INT8_GRAD) return HM_ERR_UNSUPPORTED;
  const bool pairs = op == HM_INT8_GATED || op == HM_INT8_GATED_GRAD;
  if (hm_status s = op == HM_INT8_GRAD ? check_grad(m, n, k) : pairs ? check_gated(m, n, k) : check_sizes(m, n, k)) return s;
  if (!buf || !buf_len) return HM_ERR_NULL;
  if (op != HM_INT8_GRAD) {
    if (m == 0) snprintf(buf, buf_len, "nothing");
    else say(plan_product(m, pairs ? n / 2 : n, pairs, k, op == HM_INT8_GATED_GRAD ? INT8_GRAD : INT8), pairs, m, pairs ? n / 2 : n, buf, buf_len);
    return HM_OK;
  }
  const GradPlan g = plan_grad(m, n, k);
  char dx[80] = "nothing", dw[80];
  if (m) say(g.dx, false, m, k, dx, sizeof dx);
  say(g.dw, false, n, k, dw, sizeof dw);
  snprintf(buf, buf_len, "dx %s; dw %s", dx, dw);
  return HM_OK;
}
