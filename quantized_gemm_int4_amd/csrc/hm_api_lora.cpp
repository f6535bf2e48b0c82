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

// Blocks along a contraction of `len` for `units` units: enough to fill the
// chip, each wave keeping 64 values of the axis or more.
int contraction_splits(int64_t units, int64_t len) {
  const int64_t want = (1024 + units - 1) / units, most = std::max<int64_t>(1, len / 256);
  return (int)std::max<int64_t>(1, std::min(std::min(want, most), (int64_t)16));
}

LoraWs lora_ws(const hm_lora_desc* d, int64_t m) {
  LoraWs w{};
  const int64_t L = d->num_adapters;
  w.max_units = m / kLoraUnit + std::min<int64_t>(L, m);
  w.splits = contraction_splits(std::max<int64_t>(w.max_units, 1), d->k);
  w.splits_n = contraction_splits(std::max<int64_t>(w.max_units, 1), d->n);
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t o = at;
    at = align256(at + bytes);
    return o;
  };
  w.hdr = take(256);
  w.units = take((size_t)w.max_units * 16);
  w.counts = take((size_t)L * 4);
  w.offsets = take((size_t)(L + 1) * 4);
  w.rows = take((size_t)m * 4);
  const int nb = moe_sort_blocks(m, nullptr);
  w.cnt = take(nb > 1 ? (size_t)nb * (size_t)L * 4 : 0);
  w.part = take((size_t)std::max(w.splits, w.splits_n) * (size_t)m * (size_t)d->rank * 4);
  w.total = at;
  return w;
}

hipError_t group_rows(const hm_lora_desc* d, const int32_t* ids, int64_t m, const LoraWs& w, uint8_t* ws,
                      LoraArgs* g, hipStream_t st) {
  int32_t* hdr = (int32_t*)(ws + w.hdr);
  int32_t* units = (int32_t*)(ws + w.units);
  int32_t* offsets = (int32_t*)(ws + w.offsets);
  int32_t* rows = (int32_t*)(ws + w.rows);
  hipError_t e = launch_moe_sort(ids, m, d->num_adapters, (int32_t*)(ws + w.counts), offsets, rows,
                                 (int32_t*)(ws + w.cnt), st);
  if (e == hipSuccess) e = launch_lora_units(offsets, d->num_adapters, hdr, units, st);
  g->R = LoraRows{hdr, units, offsets, rows, w.max_units};
  return e;
}

LoraArgs args_of(const hm_lora_desc* d, const uint16_t* x, const int32_t* ids, const uint16_t* a, const uint16_t* b,
                 const float* scales, int64_t m) {
  LoraArgs g{};
  g.x = x;
  g.a = a;
  g.b = b;
  g.scales = scales;
  g.ids = ids;
  g.M = m;
  g.N = d->n;
  g.K = d->k;
  g.rank = d->rank;
  g.L = d->num_adapters;
  return g;
}

}  // namespace

HM_API hm_status hm_lora_workspace_size(const hm_lora_desc* d, int64_t m, size_t* bytes) {
  if (hm_status s = check_lora(d, m)) return s;
  if (!bytes) return HM_ERR_NULL;
  *bytes = m ? lora_ws(d, m).total : 0;
  return HM_OK;
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
  const LoraWs w = lora_ws(d, m);
  if (!ws) return HM_ERR_NULL;
  if (ws_bytes < w.total) return HM_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return HM_ERR_ALIGN;
  LoraArgs g = args_of(d, x, adapter_ids, a, b, scales, m);
  g.base = base;
  g.y = y;
  g.h = h;
  g.splits = w.splits;
  g.part = (h && w.splits == 1) ? h : (float*)((uint8_t*)ws + w.part);
  hipError_t e = group_rows(d, adapter_ids, m, w, (uint8_t*)ws, &g, stream);
  if (e == hipSuccess) e = launch_lora_shrink(g, stream);
  if (e == hipSuccess) e = launch_lora_expand(g, stream);
  return e == hipSuccess ? HM_OK : HM_ERR_HIP;
}

HM_API hm_status hm_lora_grad_workspace_size(const hm_lora_desc* d, int64_t m, size_t* bytes) {
  if (hm_status s = check_lora(d, m)) return s;
  if (!bytes) return HM_ERR_NULL;
  *bytes = m ? lora_ws(d, m).total : 0;
  return HM_OK;
}

HM_API hm_status hm_lora_grad(const hm_lora_desc* d, const uint16_t* dy, const uint16_t* x, const float* h,
                              const int32_t* adapter_ids, const uint16_t* a, const uint16_t* b, const float* scales,
                              int64_t m, const uint16_t* dx_base, uint16_t* dx, uint16_t* da, uint16_t* db, void* ws,
                              size_t ws_bytes, hipStream_t stream) {
  if (hm_status s = check_lora(d, m)) return s;
  if (!da || !db) return HM_ERR_NULL;
  if (!aligned(da, 16) || !aligned(db, 16)) return HM_ERR_ALIGN;
  LoraArgs g = args_of(d, x, adapter_ids, a, b, scales, m);
  g.dy = dy;
  g.h = const_cast<float*>(h);
  g.da = da;
  g.db = db;
  if (m == 0) return launch_lora_outer(g, stream) == hipSuccess ? HM_OK : HM_ERR_HIP;
  if (!dy || !x || !h || !adapter_ids || !a || !b || !scales) return HM_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(h, 16) || !aligned(a, 16) || !aligned(b, 16) ||
      !aligned(dx_base, 16) || !aligned(dx, 16) || !aligned(adapter_ids, 4) || !aligned(scales, 4))
    return HM_ERR_ALIGN;
  const LoraWs w = lora_ws(d, m);
  if (!ws) return HM_ERR_NULL;
  if (ws_bytes < w.total) return HM_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return HM_ERR_ALIGN;
  g.base = dx_base;
  g.y = dx;
  g.splits = w.splits_n;
  g.part = (float*)((uint8_t*)ws + w.part);
  hipError_t e = group_rows(d, adapter_ids, m, w, (uint8_t*)ws, &g, stream);
  if (e == hipSuccess) e = launch_lora_shrink_b(g, stream);
  if (e == hipSuccess && dx) e = launch_lora_expand_a(g, stream);
  if (e == hipSuccess) e = launch_lora_outer(g, stream);
  return e == hipSuccess ? HM_OK : HM_ERR_HIP;
}
