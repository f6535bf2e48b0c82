// Launch shapes of the expert-order row operators and the low-rank adapters
// over their whole range of sizes: the library's own launchers, built for the
// host alone and linked with stand-ins of the few runtime functions they call.
// The stand-in of hipLaunchKernel checks each launch against the hardware's
// limits (a dimension's blocks x threads below 2^32, at most 65535 blocks
// along y, 1024 threads a block), runs nothing and touches no memory.  A call
// that the size checks accept has to be launched.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <map>
#include <string>

#include "hm.h"
#include "lora.h"

static std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
static std::map<std::string, long> g_launches;
static uintptr_t g_ws = 0, g_ws_end = 0;
static char g_what[256] = "";

static void need(bool ok, const char* what) {
  if (!ok) {
    printf("check failed: %s; call: %s\n", what, g_what);
    exit(1);
  }
}

struct Config { dim3 grid, block; size_t shared; hipStream_t stream; };
static Config g_config;

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
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t, hipStream_t) {
  const std::string& name = names().at(f);
  ++g_launches[name];
  need(grid.x >= 1 && grid.y >= 1 && grid.z == 1 && block.y == 1 && block.z == 1, "an empty launch");
  need(block.x >= 64 && block.x <= 1024 && block.x % 64 == 0, "threads of a block");
  if ((uint64_t)grid.x * block.x >= (1ull << 32)) printf("%s: %u blocks of %u\n", name.c_str(), grid.x, block.x);
  need((uint64_t)grid.x * block.x < (1ull << 32), "blocks x threads along x");
  need(grid.y <= 65535, "blocks along y");
  if (name.find("k_lora_dx") != std::string::npos) {
    // the packed g and h: their kTerms terms a value inside the workspace, apart from each other and the sums
    const auto& o = *static_cast<hm::LoraGradArgs*>(args[1]);
    const uint64_t packed = (uint64_t)o.R.max_units * hm::kTerms * hm::lora_rp(o.rank) * hm::kLoraUnit * 2;
    if (o.M) {
      need((uintptr_t)o.gt >= g_ws && (uintptr_t)o.gt + packed <= (uintptr_t)o.ht, "packed g");
      need((uintptr_t)o.ht + packed <= (o.chunks > 1 ? (uintptr_t)o.sums : g_ws_end), "packed h");
    }
  }
  return hipSuccess;
}
}

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
  const int64_t v = lo + (int64_t)(next() % (uint64_t)(top > 0 ? top : 1));
  return v > hi ? hi : v;
}

template <class T> static T* at(uint64_t slot) { return reinterpret_cast<T*>((uintptr_t)(slot << 48)); }

static void rows(int64_t t, int32_t topk, int32_t E, int64_t n) {
  auto *x = at<uint16_t>(1), *out = at<uint16_t>(2);
  auto *w = at<float>(3), *dw = at<float>(4);
  auto *ids = at<int32_t>(5), *i6 = at<int32_t>(6);
  void* ws = at<void>(7);
  snprintf(g_what, sizeof g_what, "t %lld topk %d E %d n %lld", (long long)t, topk, E, (long long)n);
  const bool ok = t >= 0 && t < (1 << 24) && n <= (1 << 24) && t * topk < (1ll << 31) && t * ((n + 511) / 512) < (1ll << 26);
  const hm_status want = ok ? HM_OK : HM_ERR_SHAPE;           // the limits that hm.h states
  need(hm_moe_collect(x, w, ids, t, topk, n, out, nullptr) == want, "collect");
  need(hm_moe_dispatch_grad(x, ids, t, topk, n, out, nullptr) == want, "dispatch gradient");
  need(hm_moe_collect_grad(x, x, w, ids, t, topk, n, out, dw, nullptr) == want, "collect gradient");
  if (topk > E) return;
  size_t bytes = 0;
  const hm_status q = hm_moe_dispatch_workspace_size(t, topk, E, &bytes);
  need(ok ? q == HM_OK : true, "size query");
  need(hm_moe_dispatch(x, ids, t, topk, E, n, out, i6, i6 + (1 << 20), i6 + (2 << 20), i6 + (3 << 20), ws, bytes, nullptr) ==
           want, "dispatch");
}

static void lora(int64_t m, int32_t rank, int32_t L, int64_t n, int64_t k, int i) {
  auto *x = at<uint16_t>(1), *a = at<uint16_t>(2), *b = at<uint16_t>(3), *base = at<uint16_t>(4), *y = at<uint16_t>(5),
       *dy = at<uint16_t>(6), *da = at<uint16_t>(7), *db = at<uint16_t>(8);
  auto *h = at<float>(9), *sc = at<float>(10);
  auto* ids = at<int32_t>(11);
  void* ws = at<void>(12);
  g_ws = (uintptr_t)ws;
  snprintf(g_what, sizeof g_what, "m %lld rank %d L %d n %lld k %lld", (long long)m, rank, L, (long long)n, (long long)k);
  const hm_lora_desc d = {HM_ABI_VERSION, rank, L, 0, n, k};
  size_t bytes = 0;
  hm_status q = hm_lora_workspace_size(&d, m, &bytes);
  need(q == HM_OK || q == HM_ERR_SHAPE, "size query");
  g_ws_end = g_ws + bytes;
  need(hm_lora(&d, x, ids, a, b, sc, m, i & 1 ? base : nullptr, i & 2 ? base : y, i & 4 ? h : nullptr, ws, bytes, nullptr) == q,
       "adapters");
  q = hm_lora_grad_workspace_size(&d, m, &bytes);
  need(q == HM_OK || q == HM_ERR_SHAPE, "size query");
  g_ws_end = g_ws + bytes;
  need(hm_lora_grad(&d, dy, x, h, ids, a, b, sc, m, i & 1 ? base : nullptr, i & 2 ? nullptr : y, da, db, ws, bytes, nullptr) == q,
       "adapter gradient");
}

int main() {
  // the largest token counts at both block sizes of the collect's gradient
  const int64_t most = (1ll << 26) / 5 - 1;
  rows(9000000, 1, 8, 2056);
  for (int64_t n : {1, 512, 513, 2048, 2049, 2056, 2560, 3584, 4096, 4097})
    for (int64_t t : {(int64_t)(1 << 23) - 1, (int64_t)(1 << 23), most, most + 1, (int64_t)(1 << 24) - 1, (int64_t)(1 << 24)}) rows(t, 1, 8, n);
  for (int i = 0; i < 100000; ++i) {
    rows(draw(0, 1 << 24), (int32_t)draw(1, 512), (int32_t)draw(1, 512), draw(1, 1 << 24));
    lora(draw(0, 1 << 20), 8 * (int32_t)draw(1, 16), (int32_t)draw(1, 512), draw(1, 1 << 24), 128 * draw(1, 8192), i);
  }
  long total = 0;
  for (const auto& k : g_launches) total += k.second;
  need(g_launches.size() > 40 && total > 100000, "launches of every kernel");
  // every kernel of these operators is reached by some size; hm_moe_sort and the grouped GEMM have the others of k_moe
  for (const auto& k : names()) {
    const std::string& s = k.second;
    if (s.find("k_moe_sortEPK") != s.npos || s.find("k_moe_sort_placeILb0") != s.npos || s.find("k_moe_schedule") != s.npos) continue;
    if (!g_launches.count(s)) printf("never launched: %s\n", s.c_str());
    need(g_launches.count(s) != 0, "a kernel that no call reaches");
  }
  printf("launch shapes ok: %ld launches of %zu kernels\n", total, g_launches.size());
  return 0;
}
