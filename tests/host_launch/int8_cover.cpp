// What the launches of the 8-bit integer layers cover: for calls over the whole range of sizes, every
// launch's blocks, tiles, groups and parts are those that its kernel (known by its template arguments) needs for
// exactly the call's output, none missing and none empty, and its operands are the call's arrays in full.  The library's own
// entry points and launchers, built for the host alone and linked with stand-ins of the runtime
// functions they call; nothing runs on a device and no memory is touched.
//
//   int8_cover           the sweep
//   int8_cover NAME      the same with one launch argument of that kernel spoilt before it is looked at: has to fail
#include <cxxabi.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <map>
#include <string>
#include <vector>

#include "hm.h"
#include "i8.h"

static std::string g_spoil;
static char g_what[256] = "";
static long g_checked = 0;

static void need(bool ok, const char* what) {
  ++g_checked;
  if (!ok) {
    printf("check failed: %s; call: %s\n", what, g_what);
    exit(1);
  }
}
static int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A kernel: its name and template arguments.
struct Kernel {
  std::string name;
  std::vector<std::string> args;
  int num(size_t i) const { return args.at(i) == "true" ? 1 : args.at(i) == "false" ? 0 : atoi(args.at(i).c_str()); }
};
static std::map<const void*, Kernel>& kernels() {
  static std::map<const void*, Kernel> m;
  return m;
}
static Kernel parse(const char* mangled) {
  int status = 0;
  char* text = abi::__cxa_demangle(mangled, nullptr, nullptr, &status);
  const std::string s = status == 0 ? text : mangled;
  free(text);
  Kernel k;
  size_t at = s.find("k_i8_"), end = s.find_first_of("<(", at);
  if (at == s.npos || end == s.npos) return k;
  k.name = s.substr(at, end - at);
  if (s[end] == '<') {
    std::string one;
    for (size_t i = end + 1; i < s.size() && s[i] != '>'; ++i) {
      if (s[i] == ',') {
        k.args.push_back(one);
        one.clear();
      } else if (s[i] != ' ') {
        one += s[i];
      }
    }
    k.args.push_back(one);
  }
  return k;
}

// The call that launches belong to.
static struct {
  int64_t m, n, k;
  int op;
  const void *x8, *w8, *xs, *ws, *dy, *out, *dw;
} g_call;
static hm::I8Copies g_copies;
static hm::TilePlan g_cut;               // the last tile launch whose parts are to be joined
static bool g_join = false;

// The output of the call that a launch with this `out` computes, and its operands.
static bool check_args(const hm::TileArgs& a, int epi) {
  const auto& c = g_call;
  const bool pairs = c.op == HM_INT8_GATED || c.op == HM_INT8_GATED_GRAD;
  if (c.op != HM_INT8_GRAD) {
    need(epi == c.op, "epilogue");
    need(a.out == c.out && a.rows == c.m && a.cols == (pairs ? c.n / 2 : c.n), "output");
    need(a.p == c.w8 && a.p_ld == c.k && a.p_bytes == a.cols * c.k && a.ps == c.ws, "weights");
    need(a.q == c.x8 && a.q_ld == c.k && a.q_bytes == c.m * c.k && a.qs == c.xs, "rows");
    need(a.kbytes == c.k && (c.op != HM_INT8_GATED_GRAD || a.dh == c.dy), "contraction");
    return pairs;
  }
  const bool dx = a.out == c.out;
  need(epi == hm::EPI_ROUND && (dx || a.out == c.dw), "one of the gradients");
  need(a.rows == (dx ? c.m : c.n) && a.cols == c.k, "output");
  const int64_t terms = dx ? c.n : c.m;
  const void* codes = dx ? c.w8 : c.x8;
  const hm::I8Copies& k = g_copies;
  const int i = dx ? 0 : 1;
  if (a.p == codes) {
    need(a.p_ld == c.k && a.p_bytes == terms * c.k && a.ps == (dx ? c.ws : c.xs) && a.terms == terms, "codes");
  } else if (terms) {
    need(a.p == (const uint8_t*)k.out[i] && k.rows[i] == terms && k.kc * 16 == c.k && k.q[i] == codes && k.s[i] == (dx ? c.ws : c.xs), "copy of the codes");
    need(a.p_ld == 2 * c.k && a.p_bytes == terms * 2 * c.k, "copy of the codes");
  }
  const int64_t ld = (c.n + 7) / 8 * 8;
  if (c.m && ld != c.n) need(a.q == (const uint8_t*)k.pad && k.dy == c.dy && k.m == c.m && k.n == c.n && k.nc * 8 == ld, "padded copy of dy");
  else if (c.m) need(a.q == (const uint8_t*)c.dy, "dy");
  need(a.q_ld == 2 * ld && a.q_bytes == 2 * c.m * ld && a.kbytes == (dx ? 2 * ld : 2 * c.m), "dy");
  return false;
}

extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* h; return &h; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, dim3*, dim3*, int*) {
  kernels()[host] = parse(name);
}
static struct { dim3 grid, block; size_t shared; hipStream_t stream; } g_config;
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
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) { return hipSuccess; }
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t shared, hipStream_t) {
  const Kernel& k = kernels().at(f);
  const bool spoil = k.name == g_spoil;
  need(!g_join || k.name == "k_i8_finish", "parts are joined next");
  if (k.name == "k_i8_few") {
    const int MB = k.num(0), NB = k.num(1), S = k.num(2), epi = k.num(3);
    const auto& a = *static_cast<hm::TileArgs*>(args[0]);
    const bool pairs = check_args(a, epi);
    const int64_t groups = *static_cast<int*>(args[2]), per = *static_cast<int*>(args[3]), width = 16 * (pairs ? NB / 2 : NB);
    int64_t total = *static_cast<uint32_t*>(args[1]);
    if (spoil) total -= groups;                    // a block of columns less
    need(per % 16 == 0 && per >= 16 && per <= 16 * MB && groups == up(a.rows, per), "groups of rows");
    need(NB >= (pairs ? 2 : 1) && (!pairs || NB % 2 == 0) && total == up(a.cols, width) * groups, "blocks of columns");
    const int own = S * (NB + MB) * 2048 > NB * MB * 1024 ? S * (NB + MB) * 2048 : NB * MB * 1024;
    need(grid.x == 8 * up(total, 8) && block.x == 256 && shared == (size_t)4 * own, "launch");
  } else if (k.name == "k_i8_few_dx") {
    const int QB = k.num(0), W = k.num(1);
    const auto& a = *static_cast<hm::TileArgs*>(args[0]);
    check_args(a, hm::EPI_ROUND);
    need(a.out == g_call.out && a.p == g_call.w8, "dx from the codes");
    int64_t total = *static_cast<uint32_t*>(args[1]);
    const int64_t groups = *static_cast<int*>(args[2]);
    if (spoil) total -= a.cols / 64;               // a group of rows less
    need(a.cols % 64 == 0 && groups == up(a.rows, 32 * QB) && total == a.cols / 64 * groups, "groups and columns");
    const int step = 4096 + QB * 4096 + 256, own = step > QB * 8192 ? step : QB * 8192;
    need(grid.x == 8 * up(total, 8) && (int)block.x == 64 * W && shared == (size_t)W * own, "launch");
  } else if (k.name == "k_i8_tile") {
    const int pm = k.num(1), epi = k.num(3), ST = k.num(4);
    const auto& a = *static_cast<hm::TileArgs*>(args[0]);
    hm::TilePlan pl = *static_cast<hm::TilePlan*>(args[1]);
    const bool pairs = check_args(a, epi);
    if (spoil) --pl.tiles_p;                       // a column of tiles less
    need((pm == 0) == (g_call.op != HM_INT8_GRAD) && (pm == 1) == (g_call.op == HM_INT8_GRAD && a.p == (a.out == g_call.out ? g_call.w8 : g_call.x8)),
         "how P is held");
    need(k.num(2) == (g_call.op == HM_INT8_GRAD && a.out == g_call.dw), "how Q is held");
    need(pl.tiles_p == up(a.cols, pairs ? 64 : 128) && pl.tiles_q == up(a.rows, 128), "tiles");
    const int64_t rest = (int64_t)pl.tiles_p * pl.tiles_q - pl.full, steps = up(a.kbytes, 128);
    need(pl.full >= 0 && rest >= 0 && (rest ? pl.cut > 1 : pl.cut == 1), "cut tiles");
    if (rest) need((int64_t)pl.cut * pl.per >= steps && (int64_t)(pl.cut - 1) * pl.per < steps, "parts");
    need(grid.x == 8 * up(pl.full, 8) + 8 * up(rest * pl.cut, 8), "blocks");
    need((ST == 2) == (pl.two == 1) && block.x == (ST == 4 ? 320 : 256), "stages");
    g_join = rest > 0;
    g_cut = pl;
  } else if (k.name == "k_i8_finish") {
    const int epi = k.num(1);
    const auto& a = *static_cast<hm::TileArgs*>(args[0]);
    const auto& pl = *static_cast<hm::TilePlan*>(args[1]);
    const bool pairs = check_args(a, epi);
    const int64_t rest = (int64_t)pl.tiles_p * pl.tiles_q - pl.full;
    const int64_t blocks = grid.x - (spoil ? 1 : 0);
    need(g_join && pl.part == g_cut.part && pl.full == g_cut.full && pl.cut == g_cut.cut && pl.tiles_p == g_cut.tiles_p && pl.tiles_q == g_cut.tiles_q,
         "the parts that were written");
    need(blocks == rest * (pairs ? 8 : 16) && block.x == 256, "blocks");
    g_join = false;
  } else if (k.name == "k_i8_big") {
    const int epi = k.num(3);
    const auto& a = *static_cast<hm::TileArgs*>(args[0]);
    const bool pairs = check_args(a, epi), grad = g_call.op == HM_INT8_GRAD;
    int64_t tp = *static_cast<int*>(args[1]), tq = *static_cast<int*>(args[2]);
    if (spoil) --tp;
    need(tp == up(a.cols, pairs ? 128 : 256) && tq == up(a.rows, 256), "tiles");
    need(k.num(1) == grad && k.num(2) == (grad && a.out == g_call.dw) && !(grad && (a.p == g_call.w8 || a.p == g_call.x8)), "how P and Q are held");
    need(grid.x == (tp * tq < 256 ? 8 * up(tp * tq, 8) : 256) && block.x == 256, "blocks");
  } else if (k.name == "k_i8_copies") {
    g_copies = *static_cast<hm::I8Copies*>(args[0]);
    if (spoil) g_copies.rows[0] -= g_copies.rows[0] > 0, g_copies.rows[1] -= g_copies.rows[1] > 0, g_copies.m -= g_copies.nc > 0;
    need(grid.x >= 1 && block.x == 256, "launch");
  } else if (k.name == "k_i8_quant_rows") {
    const int CH = k.num(0), W = k.num(1);
    const int64_t m = *static_cast<int64_t*>(args[1]), n = *static_cast<int64_t*>(args[2]);
    const int64_t width = 512ll * CH * W - (spoil ? 512 * CH * W - 1 : 0);
    need(m == g_call.m && n == g_call.k && n <= width && block.x == 256, "a row in the registers");
    need(grid.x >= 1 && grid.x <= 65536 && (grid.x == 65536 || (int64_t)grid.x * 4 / W >= m), "rows");
  } else {
    need(k.name == "k_i8_quant_long_rows" && block.x == 256, "a kernel known here");
  }
  return hipSuccess;
}
}

static uint64_t g_rng = 7;
static uint64_t next() {
  g_rng ^= g_rng << 13;
  g_rng ^= g_rng >> 7;
  g_rng ^= g_rng << 17;
  return g_rng;
}
// Of 1..hi: over the logarithm, and often next to a multiple of 128.
static int64_t draw(int64_t hi) {
  int bits = 1;
  while ((hi >> bits) > 0) ++bits;
  int64_t v = 1 + (int64_t)(next() % (1ull << (1 + next() % bits)));
  if (next() % 3 == 0) v = (v + 127) / 128 * 128 + (int64_t)(next() % 5) - 2;
  return v < 1 ? 1 : v > hi ? hi : v;
}

template <class T> static T* at(uint64_t slot) { return reinterpret_cast<T*>((uintptr_t)(slot << 44)); }

static void call(int64_t m, int64_t n, int64_t k) {
  auto *x8 = at<int8_t>(1), *w8 = at<int8_t>(2);
  auto *xs = at<float>(3), *wsc = at<float>(4);
  auto *dy = at<uint16_t>(5), *out = at<uint16_t>(6), *dw = at<uint16_t>(7);
  void* ws = at<void>(8);
  snprintf(g_what, sizeof g_what, "m %lld n %lld k %lld", (long long)m, (long long)n, (long long)k);
  size_t b = 0;
  auto begin = [&](int op) {
    g_call = {m, n, k, op, x8, w8, xs, wsc, dy, out, dw};
    g_copies = hm::I8Copies{};
  };
  auto end = [&](hm_status s) { need(s == HM_OK && !g_join, "call"); };
  if (hm_gemm_int8_workspace_size(m, n, k, &b) != HM_OK) return;
  begin(HM_INT8_GEMM);
  end(hm_gemm_int8(x8, xs, w8, wsc, m, n, k, out, ws, b, nullptr));
  if (n % 2 == 0) {
    begin(HM_INT8_GATED);
    end(hm_gemm_int8_gated_workspace_size(m, n, k, &b));
    end(hm_gemm_int8_gated(x8, xs, w8, wsc, m, n, k, out, ws, b, nullptr));
    begin(HM_INT8_GATED_GRAD);
    end(hm_gemm_int8_gated_grad_workspace_size(m, n, k, &b));
    end(hm_gemm_int8_gated_grad(dy, x8, xs, w8, wsc, m, n, k, out, ws, b, nullptr));
  }
  if (hm_gemm_int8_grad_workspace_size(m, n, k, &b) != HM_OK) return;
  for (int want = 1; want < 4; ++want) {
    begin(HM_INT8_GRAD);
    end(hm_gemm_int8_grad(dy, x8, xs, w8, wsc, m, n, k, want & 1 ? out : nullptr, want & 2 ? dw : nullptr, ws, b, nullptr));
  }
}

int main(int argc, char** argv) {
  if (argc > 1) g_spoil = argv[1];
  for (int64_t m : {0, 1, 15, 16, 17, 127, 128, 129, 1024, 1025, 8388480})
    for (int64_t n : {1, 2, 127, 128, 129, 258, 1 << 22})
      for (int64_t k : {128, 256, 130944}) call(m, n, k);
  for (int i = 0; i < 40000; ++i) call(draw(8388480), draw(1 << 22), 128 * (1 + (int64_t)(next() % 1023)));
  for (int i = 0; i < 80000; ++i) call(draw(10000), draw(40000), 128 * draw(128));
  for (int i = 0; i < 10000; ++i) {
    const int64_t m = draw(1 << 24), k = draw(32768);
    g_call = {m, 0, k, -1};
    need(hm_quant_int8_rows(at<uint16_t>(1), m, k, at<int8_t>(2), at<float>(3), nullptr) == HM_OK, "rows");
  }
  printf("int8 cover ok: %ld checks\n", g_checked);
  return 0;
}
