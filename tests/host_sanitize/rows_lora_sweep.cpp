// Sweep of the host code of the expert-order row operators and the low-rank
// adapters (hm_api_rows.cpp, hm_api_lora.cpp) under AddressSanitizer and
// UndefinedBehaviorSanitizer.  The kernel launchers are checking stand-ins:
// each checks the arguments against what its kernel assumes (every workspace
// range inside the caller's bytes, launch shapes within the hardware's
// limits) and touches no memory.  A call has to succeed exactly when its size
// query does, and to fail with one workspace byte less.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "hm.h"
#include "lora.h"

static uintptr_t g_ws = 0, g_ws_end = 0;
static long g_launches = 0, g_calls = 0;

static void need(bool ok, const char* what) {
  if (!ok) {
    fprintf(stderr, "check failed: %s\n", what);
    exit(1);
  }
}
static bool in_ws(const void* p, uint64_t bytes) {
  return bytes == 0 || ((uintptr_t)p >= g_ws && (uintptr_t)p + bytes <= g_ws_end);
}

namespace hm {

hipError_t launch_moe_sort_pos(const int32_t*, int64_t P, int E, int32_t*, int32_t*, int32_t*, int32_t* positions,
                               int32_t* cnt, hipStream_t) {
  const int nb = moe_sort_blocks(P, nullptr);
  need(positions && P > kSortDispatch && E >= 1 && E <= 512, "chunked sort");
  need(nb > 1 && in_ws(cnt, (uint64_t)nb * E * 4), "chunk counts in the workspace");
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_dispatch_small(const uint16_t* x, const int32_t*, int64_t t, int topk, int E, int64_t n, uint16_t*,
                                 int32_t*, int32_t*, int32_t*, int32_t*, hipStream_t) {
  need(x && t >= 1 && t * topk <= kSmallPairs && kSmallPairs <= 1024 && E <= 512 && n >= 1, "one-launch dispatch");
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_dispatch_sort(const int32_t*, int64_t P, int E, int32_t*, int32_t*, int32_t*, int32_t*, hipStream_t) {
  need(P >= 1 && P <= kSortDispatch && E <= 512, "one-launch sort");
  ++g_launches;
  return hipSuccess;
}
static void rows_grid(int64_t t, int topk, int64_t n) {
  need(t >= 1 && topk >= 1 && t * topk < (1ll << 31) && n >= 1, "rows");
  need((t * ((n + 511) / 512) + 3) / 4 < (1ll << 24) && t < (1ll << 24), "blocks of a launch");
  ++g_launches;
}
hipError_t launch_dispatch_rows(const uint16_t*, const int32_t*, int64_t t, int topk, int64_t n, uint16_t*, hipStream_t) {
  rows_grid(t, topk, n);
  return hipSuccess;
}
hipError_t launch_collect(const uint16_t*, const float*, const int32_t*, int64_t t, int topk, int64_t n, uint16_t*,
                          hipStream_t) {
  rows_grid(t, topk, n);
  return hipSuccess;
}
hipError_t launch_collect_grad(const uint16_t*, const uint16_t*, const float*, const int32_t*, int64_t t, int topk,
                               int64_t n, uint16_t*, float*, hipStream_t) {
  rows_grid(t, topk, n);
  return hipSuccess;
}

static void check_rows(const LoraRows& R, int64_t M, int L) {
  need(R.unit_rows == 16 || R.unit_rows == 32 || R.unit_rows == 64, "unit rows");
  need(R.max_units >= M / R.unit_rows + (L < M ? L : M), "units for every split of the rows");
  need(in_ws(R.units, (uint64_t)R.max_units * 8) && in_ws(R.first, (uint64_t)(L + 1) * 4) &&
           in_ws(R.rows, (uint64_t)R.max_units * R.unit_rows * 4), "grouping in the workspace");
}
static void check_lora(const LoraArgs& g, bool direct, bool trans) {
  const int rp = lora_rp(g.rank), unit = direct ? 16 : g.R.unit_rows;
  need(g.z && g.a && g.b && g.scales && g.ids && g.M >= 1 && g.M <= kLoraMaxRows, "arguments");
  need(g.rank % 8 == 0 && g.rank >= 8 && g.rank <= rp && rp <= 128 && g.K % 128 == 0, "ranks and steps");
  need(!direct || (!trans && g.M <= kLoraDirect), "direct calls are small");
  need(!trans || unit == kLoraUnit, "units of the gradient");
  need(g.splits >= 1 && g.splits <= lora_max_splits(rp, unit, trans), "splits the expansion adds");
  need(g.part == g.h ? g.splits == 1 : in_ws(g.part, (uint64_t)g.splits * g.M * g.rank * 4), "contracted values in the workspace");
  if (!direct) check_rows(g.R, g.M, g.L);
}
hipError_t launch_lora_plan(const int32_t* ids, int64_t M, int L, int unit_rows, int64_t max_units, int32_t* units,
                            int32_t* rows, int32_t* first, hipStream_t) {
  need(ids != nullptr && M >= 1, "ids");
  check_rows(LoraRows{units, rows, first, max_units, unit_rows}, M, L);
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_lora_shrink(const LoraArgs& g, bool direct, bool trans, hipStream_t) {
  check_lora(g, direct, trans);
  need((direct ? g.M : g.R.max_units * (g.R.unit_rows == 64 ? 2 : 1)) <= 65535, "grid of the contraction");
  ++g_launches;
  return hipSuccess;
}
static int64_t check_expand(const LoraArgs& g, bool direct, bool trans) {
  check_lora(g, direct, trans);
  const int64_t cols = trans ? g.K : g.N, unit = direct ? 16 : g.R.unit_rows;
  need(g.y != nullptr && g.group >= 1 && g.cols >= kLoraCols && g.cols % kLoraCols == 0, "blocks of the expansion");
  need(unit == 64 ? g.cols == kLoraCols : g.group == 1, "units of few rows come one to a block, others against one part");
  const int64_t per = (cols + 8 * g.cols - 1) / (8 * g.cols);
  const int64_t groups = direct ? g.M : (g.R.max_units + g.group - 1) / g.group + (g.M + 63) / 64;
  return 8 * per * groups;
}
hipError_t launch_lora_expand(const LoraArgs& g, bool direct, hipStream_t) {
  need(check_expand(g, direct, false) < (1ll << 24), "grid of the expansion");
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_lora_small(const LoraArgs& g, int parts, hipStream_t) {
  need(g.M >= 1 && g.M <= 16 && g.rank <= 64 && parts >= 1 && parts * g.M <= 256 && g.y, "one-launch call");
  ++g_launches;
  return hipSuccess;
}
static void check_grad(const LoraGradArgs& g) {
  const uint64_t packed = (uint64_t)g.R.max_units * 2 * lora_rp(g.rank) * kLoraUnit * 2;
  check_rows(g.R, g.M, g.L);
  need(in_ws(g.gt, packed) && in_ws(g.ht, packed) && g.chunks >= 1 && g.chunks <= 16, "packed values in the workspace");
  need(g.chunks == 1 || in_ws(g.sums, 2ull * g.chunks * g.rank * (g.K + g.N) * 4), "partial sums in the workspace");
  need(in_ws(g.part, (uint64_t)g.splits * g.M * g.rank * 4), "g in the workspace");
}
hipError_t launch_lora_dx(const LoraArgs& g, const LoraGradArgs& o, hipStream_t) {
  need(o.da && o.db && o.L >= 1 && o.L <= 512, "outputs of the zeros");
  int64_t blocks = o.L * lora_zero_parts(o.rank, o.K, o.N) + 8;
  if (o.M) {
    check_grad(o);
    blocks += 4 * o.R.max_units + 8 + (g.y ? check_expand(g, false, true) : 0);
  }
  need(blocks < (1ll << 24), "grid of the dx launch");
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_lora_outer(const LoraGradArgs& g, hipStream_t) {
  check_grad(g);
  const int64_t per = ((g.N + 127) / 128 + g.K / 128 + 7) / 8, rp = lora_rp(g.rank);
  need(8 * per * g.chunks * (rp == 16 ? 1 : rp / 32) < (1ll << 24), "grid of the outer products");
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_lora_sums(const LoraGradArgs& g, hipStream_t) {
  check_grad(g);
  need(g.da && g.db && g.L >= 1 && g.L <= 512 && g.chunks > 1, "sums");
  ++g_launches;
  return hipSuccess;
}

}  // namespace hm

static uint64_t g_rng = 1;
static int64_t draw(int64_t lo, int64_t hi) {                 // inclusive, splitmix64; over the logarithm
  auto next = [] {
    g_rng += 0x9E3779B97F4A7C15ull;
    uint64_t z = g_rng;
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
  };
  int bits = 0;
  while ((hi >> bits) > 0) ++bits;
  const int64_t top = 1ll << (next() % (uint64_t)(bits + 1));
  int64_t v = lo + (int64_t)(next() % (uint64_t)(top > 0 ? top : 1));
  return v > hi ? hi : v;
}

template <class T> static T* dev(uint64_t slot) { return reinterpret_cast<T*>((uintptr_t)0x7f0000000000ull + slot * 0x10000000000ull); }

int main() {
  auto *bf = dev<uint16_t>(1), *out = dev<uint16_t>(2);
  auto* f = dev<float>(3);
  auto* ids = dev<int32_t>(4);
  void* ws = dev<void>(8);
  g_ws = (uintptr_t)ws;
  for (int i = 0; i < 200000; ++i) {
    hm_lora_desc d = {HM_ABI_VERSION, (int32_t)(8 * draw(1, 16)), (int32_t)draw(1, 512), 0, draw(1, 1 << 24), 128 * draw(1, 8192)};
    const int64_t m = draw(0, 1 << 20);
    for (int grad = 0; grad < 2; ++grad) {
      size_t bytes = 0;
      const hm_status q = grad ? hm_lora_grad_workspace_size(&d, m, &bytes) : hm_lora_workspace_size(&d, m, &bytes);
      auto call = [&](size_t b) {
        g_ws_end = g_ws + b;
        ++g_calls;
        if (grad) return hm_lora_grad(&d, bf, bf, f, ids, bf, bf, f, m, bf, i % 3 ? out : nullptr, out, out, ws, b, nullptr);
        return hm_lora(&d, bf, ids, bf, bf, f, m, i % 5 ? bf : nullptr, out, i % 2 ? f : nullptr, ws, b, nullptr);
      };
      need(q == HM_OK || q == HM_ERR_SHAPE, "a size or a refusal");
      need(call(bytes) == q, "the call agrees with its size query");
      if (q == HM_OK && bytes) need(call(bytes - 1) == HM_ERR_WORKSPACE, "one byte less is refused");
    }
    const int64_t t = draw(0, 1 << 24), n = draw(1, 1 << 24);
    const int32_t topk = (int32_t)draw(1, 512), E = (int32_t)draw(1, 520);
    size_t bytes = 0;
    const hm_status q = hm_moe_dispatch_workspace_size(t, topk, E, &bytes);
    g_ws_end = g_ws + bytes;
    const hm_status c = hm_moe_dispatch(bf, ids, t, topk, E, n, out, ids, ids, ids, ids, ws, bytes, nullptr);
    need(q == HM_OK ? c == HM_OK || c == HM_ERR_SHAPE : c == q, "dispatch agrees with its size query");
    const hm_status a = hm_moe_collect(bf, f, ids, t, topk, n, out, nullptr);
    need(hm_moe_dispatch_grad(bf, ids, t, topk, n, out, nullptr) == a, "one rule for the rows");
    need(hm_moe_collect_grad(bf, bf, f, ids, t, topk, n, out, f, nullptr) == a, "one rule for the rows");
    if (c == HM_OK && t) need(a == HM_OK, "what can be dispatched can be collected");
  }
  need(g_launches > 100000, "launches happened");
  printf("rows and adapters sweep ok: %ld adapter calls, %ld launches\n", g_calls, g_launches);
  return 0;
}
