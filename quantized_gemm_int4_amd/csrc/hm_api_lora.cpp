// C ABI entry points of the low-rank adapters: argument checks, workspace
// layout and launches.  Every check runs before any launch; nothing is
// allocated.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/hm.h"
#include "lora.h"

#define HM_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace hm;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Whether an output's bytes and those of one of the arrays it must leave alone
// meet.  No array is longer than the card's memory (288 GB), so lengths end
// at 2^39 and ends do not wrap.
struct Span {
  const void* p;             // null: no array
  uint64_t bytes;
};
bool meets(const Span& out, const Span& in) {
  if (!out.p || !in.p) return false;
  constexpr uint64_t kMost = 1ull << 39;
  const uint64_t a = (uintptr_t)out.p, b = (uintptr_t)in.p;
  return a < b + std::min(in.bytes, kMost) && b < a + std::min(out.bytes, kMost);
}
template <size_t N> bool meets_any(const Span& out, const Span (&in)[N]) {
  return std::any_of(in, in + N, [&](const Span& s) { return meets(out, s); });
}

hm_status check_lora(const hm_lora_desc* d, int64_t m) {
  if (!d) return HM_ERR_NULL;
  if (d->abi != HM_ABI_VERSION) return HM_ERR_ABI;
  if (d->rank < 8 || d->rank > 128 || (d->rank % 8) != 0 || d->num_adapters < 1 || d->num_adapters > 512 ||
      d->reserved != 0)
    return HM_ERR_SHAPE;
  if (d->n < 1 || d->n > (1ll << 24) || d->k < 128 || (d->k % 128) != 0 || d->k > (1ll << 20)) return HM_ERR_SHAPE;
  if (m < 0 || m > kLoraMaxRows) return HM_ERR_SHAPE;
  return HM_OK;
}

// Blocks of one launch stay under 2^24 (2^32 threads).
constexpr int64_t kMaxBlocks = (1ll << 24) - 1;

// Calls that run both products in one launch: up to 16 rows, and an A (of
// padded rank) that every block can read by itself.  One launch against two,
// and as a Python loop issues them (the host needs 3 us a launch): m = 1, k =
// 2048, n = 7168, rank 16 6.9 against 7.8 us, 8.5 against 10.7; m = 8, k = 4096,
// n = 14336, rank 16 8.3 against 8.4, 8.4 against 10.9; beyond: rank 64 (262144
// values) 16.5 against 10.3, m = 48 14.3 against 12.5.
constexpr int64_t kSmallA = 131072;
constexpr int64_t kSmallRows = 16;

// Byte offsets in the workspace (total a multiple of 256) and launch shape.
struct LoraPlan {
  size_t units, rows, first, part, gt, ht, sums, total;
  int64_t max_units;
  int unit_rows, splits, group, cols, chunks;
  int parts;                 // column parts of the one-launch kernel, 0: not taken
  bool direct;
};

// Rows per unit: 64 where the adapters can have that many rows each on average
// (every loaded value of A and B then serves four MFMAs), fewer where units
// would be mostly empty: m = 256, 32 adapters of rank 64, k = 7168, n = 4096
// 22.6 us with 16 rows, 26.8 with 64; m = 128, 40 of rank 128, k = 4096, n =
// 7168 39.7 against 45.0.  The rule sees the adapters that are loaded, not those
// in use, which can go either way: with 6 of 512 in use, m = 8192, k = 4096, n =
// 14336, rank 64 takes 231 us where 64-row units would take 169 (6 loaded: 148);
// with 7 of 64, m = 1021, k = 7168, n = 4099 36.5 against 28.1; with 4 of 512,
// m = 256, k = 7168, n = 4096 27.4 against 36.3.
int rows_per_unit(int64_t m, int64_t L) { return m <= 16 * L ? 16 : (m <= 32 * L ? 32 : 64); }

hm_status plan_lora(const hm_lora_desc* d, int64_t m, bool grad, LoraPlan* out) {
  LoraPlan w{};
  const int64_t L = d->num_adapters, len = grad ? d->n : d->k, cols = grad ? d->k : d->n;
  w.direct = !grad && m <= kLoraDirect;
  w.unit_rows = grad ? kLoraUnit : (w.direct ? 16 : rows_per_unit(m, L));
  w.max_units = w.direct ? m : m / w.unit_rows + std::min<int64_t>(L, m);
  // blocks along the contraction: about 4096 waves in all (16-row units) or
  // 640 blocks (32-row blocks; m = 8192, rank 64: 1024 blocks cost 3 us more, a gradient of rank 32 12 us, in
  // sums that are read again), each wave keeping a step of 64 or more
  const bool few = w.unit_rows == 16;
  const int rp = lora_rp(d->rank);
  const int64_t blocks = few ? w.max_units : w.max_units * (w.unit_rows / 32);
  const int64_t waves = lora_waves(rp, w.unit_rows, grad);
  const int64_t want = few ? 4096 / (blocks * waves) : 640 / blocks;
  const int64_t most = std::min<int64_t>(lora_max_splits(rp, w.unit_rows, grad), len / (64 * waves));
  w.splits = (int)std::max<int64_t>(1, std::min(want, most));
  // expanding blocks: two units against one part of B where there are many (m = 8192, n = 14336, rank 64: 148 us, 154
  // with one, 152 with four; rank 16: 116, 113, 119), several parts of the columns where there are many units of few
  // rows (rank 16: m = 48, n = 14336 12.6 us, 13.0 with one part; m = 128 24.1 against 28.0; m = 32, n = 28672 17.2
  // against 18.3; rank 64, m = 64 31.8 against 31.3; where one adapter has all 64 rows 12.3 against 10.5)
  int64_t slabs = 8 * ((cols + 8 * kLoraCols - 1) / (8 * kLoraCols));
  w.group = w.direct || w.unit_rows < 64 ? 1 : (w.max_units * slabs >= 2048 ? 2 : 1);
  w.cols = kLoraCols;
  while (few && w.max_units * slabs > 2048 && w.cols < 4 * kLoraCols && cols > 8 * w.cols) {
    w.cols *= 2;
    slabs = 8 * ((cols + 8 * w.cols - 1) / (8 * w.cols));
  }
  int64_t launch = slabs * ((w.max_units + w.group - 1) / w.group + (m + 63) / 64);
  if (grad) launch += 4 * w.max_units + L * lora_zero_parts(d->rank, d->k, d->n) + 16;
  if (launch > kMaxBlocks) return HM_ERR_SHAPE;
  if (!grad && m <= kSmallRows && d->rank <= 64 && (int64_t)lora_rp(d->rank) * d->k <= kSmallA) {
    const int64_t waves = d->rank > 32 ? 8 : 16, most = (d->n + 64 * waves - 1) / (64 * waves);
    w.parts = (int)std::max<int64_t>(1, std::min<int64_t>(most, 256 / m));
    *out = w;
    return HM_OK;
  }
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t o = at;
    at = align256(at + bytes);
    return o;
  };
  if (!w.direct) {
    w.units = take((size_t)w.max_units * 8);
    w.rows = take((size_t)w.max_units * (size_t)w.unit_rows * 4);
    w.first = take((size_t)(L + 1) * 4);
  }
  w.part = take((size_t)w.splits * (size_t)m * (size_t)d->rank * 4);
  if (grad) {
    const size_t packed = (size_t)w.max_units * kTerms * (size_t)lora_rp(d->rank) * kLoraUnit * 2;
    w.gt = take(packed);
    w.ht = take(packed);
    // about 768 blocks, three to a compute unit (m = 8192, k = 4096, n = 14336, rank 32: 159 us a call; 512 168, 1024
    // 165; rank 64: 231, 252, 239), a chunk of four units or more (m = 777, rank 16: 33.3 us a call; of sixteen 38.1)
    const int64_t tiles = ((d->n + 127) / 128 + d->k / 128) * std::max(1, lora_rp(d->rank) / 32);
    w.chunks = (int)std::max<int64_t>(1, std::min<int64_t>(16, std::min((767 + tiles) / tiles, w.max_units / 4)));
    w.sums = take(w.chunks > 1 ? (size_t)(2 * w.chunks) * (size_t)d->rank * (size_t)(d->k + d->n) * 4 : 0);
  }
  w.total = at;
  *out = w;
  return HM_OK;
}

hm_status workspace_size(const hm_lora_desc* d, int64_t m, bool grad, size_t* bytes) {
  if (hm_status s = check_lora(d, m)) return s;
  if (!bytes) return HM_ERR_NULL;
  LoraPlan w{};
  if (m)
    if (hm_status s = plan_lora(d, m, grad, &w)) return s;
  *bytes = w.total;
  return HM_OK;
}

hipError_t group_rows(const hm_lora_desc* d, const int32_t* ids, int64_t m, const LoraPlan& w, uint8_t* ws,
                      LoraRows* R, hipStream_t st) {
  int32_t* units = (int32_t*)(ws + w.units);
  int32_t* rows = (int32_t*)(ws + w.rows);
  int32_t* first = (int32_t*)(ws + w.first);
  *R = LoraRows{units, rows, first, w.max_units, w.unit_rows};
  return launch_lora_plan(ids, m, d->num_adapters, w.unit_rows, w.max_units, units, rows, first, st);
}

LoraArgs args_of(const hm_lora_desc* d, const uint16_t* z, const int32_t* ids, const uint16_t* a, const uint16_t* b,
                 const float* scales, int64_t m, const uint16_t* base, uint16_t* y, const LoraPlan& w, uint8_t* ws) {
  LoraArgs g{};
  g.z = z;
  g.a = a;
  g.b = b;
  g.scales = scales;
  g.ids = ids;
  g.M = m;
  g.N = d->n;
  g.K = d->k;
  g.rank = d->rank;
  g.L = d->num_adapters;
  g.base = base;
  g.y = y;
  g.part = (float*)(ws + w.part);
  g.splits = w.splits;
  g.group = w.group;
  g.cols = w.cols;
  return g;
}

}  // namespace

HM_API hm_status hm_lora_workspace_size(const hm_lora_desc* d, int64_t m, size_t* bytes) {
  return workspace_size(d, m, false, bytes);
}

HM_API hm_status hm_lora(const hm_lora_desc* d, const uint16_t* x, const int32_t* adapter_ids, const uint16_t* a,
                         const uint16_t* b, const float* scales, int64_t m, const uint16_t* base, uint16_t* y,
                         float* h, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (hm_status s = check_lora(d, m)) return s;
  if (m == 0) return HM_OK;
  if (!x || !adapter_ids || !a || !b || !scales || !y) return HM_ERR_NULL;
  if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(y, 16) || !aligned(base, 16) ||
      !aligned(h, 16) || !aligned(adapter_ids, 4) || !aligned(scales, 4))
    return HM_ERR_ALIGN;
  LoraPlan w;
  if (hm_status s = plan_lora(d, m, false, &w)) return s;
  if (w.total) {
    if (!ws) return HM_ERR_NULL;
    if (ws_bytes < w.total) return HM_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return HM_ERR_ALIGN;
  }
  const uint64_t um = m, k = d->k, n = d->n, mats = 2ull * d->num_adapters * d->rank;
  if (meets_any({y, 2 * um * n}, {{x, 2 * um * k}, {a, mats * k}, {b, mats * n}, {y == base ? nullptr : base, 2 * um * n}}))
    return HM_ERR_UNSUPPORTED;
  LoraArgs g = args_of(d, x, adapter_ids, a, b, scales, m, base, y, w, (uint8_t*)ws);
  g.h = h;
  if (w.parts) return launch_lora_small(g, w.parts, stream) == hipSuccess ? HM_OK : HM_ERR_HIP;
  if (h && w.splits == 1) g.part = h;
  hipError_t e = w.direct ? hipSuccess : group_rows(d, adapter_ids, m, w, (uint8_t*)ws, &g.R, stream);
  if (e == hipSuccess) e = launch_lora_shrink(g, w.direct, false, stream);
  if (e == hipSuccess) e = launch_lora_expand(g, w.direct, stream);
  return e == hipSuccess ? HM_OK : HM_ERR_HIP;
}

HM_API hm_status hm_lora_grad_workspace_size(const hm_lora_desc* d, int64_t m, size_t* bytes) {
  return workspace_size(d, m, true, bytes);
}

HM_API hm_status hm_lora_grad(const hm_lora_desc* d, const uint16_t* dy, const uint16_t* x, const float* h,
                              const int32_t* adapter_ids, const uint16_t* a, const uint16_t* b, const float* scales,
                              int64_t m, const uint16_t* dx_base, uint16_t* dx, uint16_t* da, uint16_t* db, void* ws,
                              size_t ws_bytes, hipStream_t stream) {
  if (hm_status s = check_lora(d, m)) return s;
  if (!da || !db) return HM_ERR_NULL;
  if (!aligned(da, 16) || !aligned(db, 16)) return HM_ERR_ALIGN;
  LoraGradArgs o{};
  o.x = x;
  o.dy = dy;
  o.h = h;
  o.M = m;
  o.N = d->n;
  o.K = d->k;
  o.rank = d->rank;
  o.L = d->num_adapters;
  o.da = da;
  o.db = db;
  if (m == 0) return launch_lora_dx(LoraArgs{}, o, stream) == hipSuccess ? HM_OK : HM_ERR_HIP;
  if (!dy || !x || !h || !adapter_ids || !a || !b || !scales) return HM_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(h, 16) || !aligned(a, 16) || !aligned(b, 16) ||
      !aligned(dx_base, 16) || !aligned(dx, 16) || !aligned(adapter_ids, 4) || !aligned(scales, 4))
    return HM_ERR_ALIGN;
  LoraPlan w;
  if (hm_status s = plan_lora(d, m, true, &w)) return s;
  if (!ws) return HM_ERR_NULL;
  if (ws_bytes < w.total) return HM_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return HM_ERR_ALIGN;
  const uint64_t um = m, k = d->k, n = d->n, mats = 2ull * d->num_adapters * d->rank;
  const Span in[] = {{dy, 2 * um * n}, {x, 2 * um * k}, {h, 4 * um * d->rank}, {a, mats * k}, {b, mats * n}};
  const Span base = {dx_base, 2 * um * k}, odx = {dx, 2 * um * k}, oda = {da, mats * k}, odb = {db, mats * n};
  if (meets_any(odx, in) || meets_any(oda, in) || meets_any(odb, in) || meets(oda, base) || meets(odb, base) ||
      (dx != dx_base && meets(odx, base)))
    return HM_ERR_UNSUPPORTED;
  uint8_t* at = (uint8_t*)ws;
  LoraArgs g = args_of(d, dy, adapter_ids, a, b, scales, m, dx_base, dx, w, at);
  hipError_t e = group_rows(d, adapter_ids, m, w, at, &g.R, stream);
  if (e == hipSuccess) e = launch_lora_shrink(g, false, true, stream);
  o.part = g.part;
  o.splits = w.splits;
  o.gt = (uint16_t*)(at + w.gt);
  o.ht = (uint16_t*)(at + w.ht);
  o.sums = (float*)(at + w.sums);
  o.chunks = w.chunks;
  o.R = g.R;
  if (e == hipSuccess) e = launch_lora_dx(g, o, stream);
  if (e == hipSuccess) e = launch_lora_outer(o, stream);
  if (e == hipSuccess && w.chunks > 1) e = launch_lora_sums(o, stream);
  return e == hipSuccess ? HM_OK : HM_ERR_HIP;
}
