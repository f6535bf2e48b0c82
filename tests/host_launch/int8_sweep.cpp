// The 8-bit integer layers over their whole range of sizes: the library's own
// entry points and launchers, built for the host alone (with sanitizers) and
// linked with stand-ins of the few runtime functions they call.  The stand-in
// of hipLaunchKernel checks each launch against the hardware's limits (blocks x
// threads below 2^32, 160 KiB of LDS) and its arguments against what the kernel
// assumes (every array of the workspace inside the caller's bytes and apart from the
// others, the parts of cut tiles covering the contraction); it runs nothing and
// touches no memory.  A call succeeds exactly when its size query does, and fails with one workspace byte less.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <map>
#include <string>

#include "hm.h"
#include "i8.h"

static std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
static std::map<std::string, long> g_launches;
static uintptr_t g_ws = 0, g_ws_end = 0;
static struct { uintptr_t from, to; } g_copies[3];
static char g_what[256] = "";

static void need(bool ok, const char* what) {
  if (!ok) {
    printf("check failed: %s; call: %s\n", what, g_what);
    exit(1);
  }
}
static bool in_ws(uintptr_t p, uint64_t bytes) { return p >= g_ws && p + bytes <= g_ws_end; }
static bool apart(uintptr_t a, uintptr_t ae, uintptr_t b, uintptr_t be) { return ae <= b || be <= a || a == ae || b == be; }

struct Config { dim3 grid, block; size_t shared; hipStream_t stream; };
static Config g_config;

static void check_tile(const std::string& name, const hm::TileArgs& a, const hm::TilePlan& pl, uint64_t blocks) {
  const bool pairs = name.find("Li1E") != name.npos || name.find("Li2EEE") != name.npos;
  (void)pairs;
  const int64_t tiles = (int64_t)pl.tiles_p * pl.tiles_q, rest = tiles - pl.full, steps = (a.kbytes + 127) / 128;
  need(pl.full >= 0 && rest >= 0 && rest < 256 && pl.cut >= 1 && pl.per >= 1, "tiles");
  need((int64_t)pl.tiles_q * 128 >= a.rows && (int64_t)(pl.tiles_q - 1) * 128 < a.rows, "tile rows");
  need(rest == 0 ? pl.cut == 1 : pl.cut > 1, "cut tiles");
  need((int64_t)pl.cut * pl.per >= steps && (int64_t)(pl.cut - 1) * pl.per < (steps ? steps : 1), "parts cover the contraction, none empty");
  need(blocks == (uint64_t)(8 * ((pl.full + 7) / 8) + 8 * ((rest * pl.cut + 7) / 8)), "blocks");
  if (rest) {
    const uintptr_t p = (uintptr_t)pl.part, e = p + (uint64_t)rest * pl.cut * 65536;
    need(in_ws(p, e - p), "parts in the workspace");
    for (const auto& c : g_copies) need(apart(p, e, c.from, c.to), "parts apart from the copies");
  }
}
static void check_operand(const hm::TileArgs& a) {
  need(a.rows >= 1 && a.cols >= 1 && a.kbytes >= 0 && a.out, "output");
  need(a.p_ld % 16 == 0 && a.q_ld % 16 == 0 && (uintptr_t)a.p % 16 == 0 && (uintptr_t)a.q % 16 == 0, "copies are 16-byte aligned");
  need(a.p_ld * 256 < (1ll << 32) && a.q_ld * 256 < (1ll << 32), "offsets in a tile fit 32 bits");
}

extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* h; return &h; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, dim3*, dim3*, int*) {
  names()[host] = name;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream) {
  g_config = {grid, block, shared, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
  *grid = g_config.grid;
  *block = g_config.block;
  *shared = g_config.shared;
  *stream = g_config.stream;
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int value) {
  need(value >= 0 && value <= 160 * 1024, "LDS of a block");
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t shared, hipStream_t) {
  const std::string& name = names().at(f);
  ++g_launches[name];
  need(grid.x >= 1 && grid.y == 1 && grid.z == 1 && block.y == 1 && block.z == 1, "an empty launch");
  need(block.x >= 64 && block.x <= 1024 && block.x % 64 == 0 && shared <= 160 * 1024, "threads and LDS of a block");
  need((uint64_t)grid.x * block.x < (1ull << 32), "blocks x threads along x");
  if (name.find("k_i8_tile") != name.npos) {
    const auto& a = *static_cast<hm::TileArgs*>(args[0]);
    check_operand(a);
    check_tile(name, a, *static_cast<hm::TilePlan*>(args[1]), grid.x);
  } else if (name.find("k_i8_finish") != name.npos) {
    const auto& pl = *static_cast<hm::TilePlan*>(args[1]);
    const uint64_t rest = (uint64_t)pl.tiles_p * pl.tiles_q - pl.full;
    need(rest >= 1 && (grid.x == rest * 8 || grid.x == rest * 16), "blocks of the last sums");
  } else if (name.find("k_i8_big") != name.npos) {
    const auto& a = *static_cast<hm::TileArgs*>(args[0]);
    const int tp = *static_cast<int*>(args[1]), tq = *static_cast<int*>(args[2]);
    check_operand(a);
    need(grid.x % 8 == 0 && grid.x <= 256 && (int64_t)tp * tq >= 1 && (int64_t)tq * 256 >= a.rows, "256 x 256 tiles");
    need(grid.x == 256 || grid.x >= (unsigned)(tp * tq), "a block for every tile");
  } else if (name.find("k_i8_few_dx") != name.npos) {
    const auto& a = *static_cast<hm::TileArgs*>(args[0]);
    const int64_t total = *static_cast<uint32_t*>(args[1]), groups = *static_cast<int*>(args[2]);
    check_operand(a);
    need(a.p_ld == a.cols && a.cols % 64 == 0 && a.terms * a.cols == a.p_bytes, "codes of the weights");
    need(groups * 128 >= a.rows && (groups - 1) * 32 < a.rows && total == a.cols / 64 * groups && grid.x >= total, "groups of rows");
  } else if (name.find("k_i8_few") != name.npos) {
    const auto& a = *static_cast<hm::TileArgs*>(args[0]);
    need(a.rows >= 1 && a.rows <= hm::kI8Few && a.kbytes % 128 == 0 && a.p_ld == a.kbytes, "few rows");
    const int64_t total = *static_cast<uint32_t*>(args[1]), groups = *static_cast<int*>(args[2]), per = *static_cast<int*>(args[3]);
    need(per % 16 == 0 && per <= 128 && groups * per >= a.rows && (groups - 1) * per < a.rows, "groups of rows, none empty");
    need(grid.x % 8 == 0 && (int64_t)grid.x >= total && total % groups == 0 && total / groups * 64 >= a.cols, "blocks of the groups");
  } else if (name.find("k_i8_copies") != name.npos) {
    const auto& c = *static_cast<hm::I8Copies*>(args[0]);
    uintptr_t from[3] = {(uintptr_t)c.out[0], (uintptr_t)c.out[1], (uintptr_t)c.pad}, to[3];
    for (int i = 0; i < 2; ++i) to[i] = from[i] + c.rows[i] * c.kc * 32;
    to[2] = from[2] + c.m * c.nc * 16;
    need(c.nc == 0 || (c.nc * 8 >= c.n && c.nc * 8 < c.n + 8), "padded rows");
    need(c.rows[0] >= 0 && c.rows[1] >= 0 && c.kc >= 8 && (to[0] > from[0] || to[1] > from[1] || to[2] > from[2]), "something to copy");
    for (int i = 0; i < 3; ++i) {
      if (to[i] == from[i]) continue;
      need(in_ws(from[i], to[i] - from[i]), "copy in the workspace");
      g_copies[i] = {from[i], to[i]};
      for (int j = 0; j < i; ++j) need(to[j] == from[j] || apart(from[i], to[i], from[j], to[j]), "copies apart");
    }
  }
  return hipSuccess;
}
}

static uint64_t g_rng = 1;
static uint64_t next() {
  g_rng += 0x9E3779B97F4A7C15ull;
  uint64_t z = g_rng;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}
static int64_t draw(int64_t lo, int64_t hi) {                 // inclusive, over the logarithm
  int bits = 0;
  while ((hi >> bits) > 0) ++bits;
  const int64_t top = 1ll << (next() % (uint64_t)(bits + 1));
  const int64_t v = lo + (int64_t)(next() % (uint64_t)(top > 0 ? top : 1));
  return v > hi ? hi : v;
}

template <class T> static T* at(uint64_t slot) { return reinterpret_cast<T*>((uintptr_t)(slot << 44)); }

static void call(int64_t m, int64_t n, int64_t k) {
  auto *x8 = at<int8_t>(1), *w8 = at<int8_t>(2);
  auto *xs = at<float>(3), *wsc = at<float>(4);
  auto *dy = at<uint16_t>(5), *out = at<uint16_t>(6), *dw = at<uint16_t>(7);
  void* ws = at<void>(8);
  g_ws = (uintptr_t)ws;
  snprintf(g_what, sizeof g_what, "m %lld n %lld k %lld", (long long)m, (long long)n, (long long)k);
  auto tiles = [](int64_t a, int64_t b) { return ((a + 127) / 128) * ((b + 127) / 128) <= (1ll << 23); };
  const bool ok = m >= 0 && m <= 8388480 && n <= (1ll << 22) && k <= 130944 && tiles(m, n);
  const hm_status want = ok ? HM_OK : HM_ERR_SHAPE;           // the limits that hm.h states
  char text[128];
  size_t bytes = 0;
  auto run = [&](hm_status expect, hm_status query, int op, auto&& go) {
    need(query == expect, "size query");
    need(hm_gemm_int8_plan(op, m, n, k, text, sizeof text) == expect, "plan");
    memset(g_copies, 0, sizeof g_copies);
    g_ws_end = g_ws + bytes;
    need(go(bytes) == expect, "call");
    if (bytes && expect == HM_OK) need(go(bytes - 1) == HM_ERR_WORKSPACE, "a byte less");
  };
  run(want, hm_gemm_int8_workspace_size(m, n, k, &bytes), HM_INT8_GEMM,
      [&](size_t b) { return hm_gemm_int8(x8, xs, w8, wsc, m, n, k, out, ws, b, nullptr); });
  const hm_status even = n % 2 ? HM_ERR_SHAPE : want;
  bytes = 0;
  run(even, hm_gemm_int8_gated_workspace_size(m, n, k, &bytes), HM_INT8_GATED,
      [&](size_t b) { return hm_gemm_int8_gated(x8, xs, w8, wsc, m, n, k, out, ws, b, nullptr); });
  bytes = 0;
  run(even, hm_gemm_int8_gated_grad_workspace_size(m, n, k, &bytes), HM_INT8_GATED_GRAD,
      [&](size_t b) { return hm_gemm_int8_gated_grad(dy, x8, xs, w8, wsc, m, n, k, out, ws, b, nullptr); });
  bytes = 0;
  const hm_status grad = ok && tiles(m, k) && tiles(n, k) ? HM_OK : HM_ERR_SHAPE;
  run(grad, hm_gemm_int8_grad_workspace_size(m, n, k, &bytes), HM_INT8_GRAD,
      [&](size_t b) { return hm_gemm_int8_grad(dy, x8, xs, w8, wsc, m, n, k, out, dw, ws, b, nullptr); });
  if (grad == HM_OK) {
    need(hm_gemm_int8_grad(dy, x8, xs, w8, wsc, m, n, k, out, nullptr, ws, bytes, nullptr) == HM_OK, "dx alone");
    need(hm_gemm_int8_grad(dy, x8, xs, w8, wsc, m, n, k, nullptr, dw, ws, bytes, nullptr) == HM_OK, "dw alone");
  }
}

int main() {
  for (int64_t m : {0, 1, 16, 64, 65, 1024, 1025, 8388480})
    for (int64_t n : {1, 2, 255, 1 << 22})
      for (int64_t k : {128, 130944}) call(m, n, k);
  for (int i = 0; i < 60000; ++i) call(draw(0, 9000000), draw(1, (1 << 22) + 100), 128 * draw(1, 1024));
  for (int i = 0; i < 60000; ++i) call(draw(0, 10000), draw(1, 40000), 128 * draw(1, 128));
  auto* x = at<uint16_t>(1);
  for (int i = 0; i < 10000; ++i) {
    const int64_t m = draw(0, 1ll << 36), k = draw(1, 1ll << 30);
    snprintf(g_what, sizeof g_what, "rows m %lld k %lld", (long long)m, (long long)k);
    const bool ok = m == 0 || k <= (1ll << 39) / m;
    need(hm_quant_int8_rows(x, m, k, at<int8_t>(2), at<float>(3), nullptr) == (ok ? HM_OK : HM_ERR_SHAPE), "rows");
  }
  long total = 0;
  for (const auto& k : g_launches) total += k.second;
  for (const auto& k : names())
    if (!g_launches.count(k.second)) printf("never launched: %s\n", k.second.c_str());
  need(g_launches.size() == names().size(), "kernels that no call reaches");
  printf("int8 sweep ok: %ld launches of %zu kernels\n", total, g_launches.size());
  return 0;
}
