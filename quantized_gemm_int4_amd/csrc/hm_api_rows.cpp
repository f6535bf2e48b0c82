// C ABI entry points of the operators on rows in expert order: argument checks
// and launches.  Every check runs before any launch; nothing is allocated.
#include <hip/hip_runtime.h>

#include "../../include/hm.h"
#include "rows.h"

#define HM_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace hm;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// A grid of `blocks` blocks of 256 threads stays under 2^32 threads.
constexpr int64_t kMaxBlocks = (1ll << 24) - 1;

hm_status check_rows(int64_t t, int32_t topk, int64_t n) {
  if (t < 0 || topk < 1 || n < 1) return HM_ERR_SHAPE;
  if (t > kMaxBlocks || t * (int64_t)topk >= (1ll << 31) || n > (1ll << 24)) return HM_ERR_SHAPE;
  if (t * ((n + 511) / 512) > 4 * kMaxBlocks) return HM_ERR_SHAPE;        // a wave per 512 columns of a row
  return HM_OK;
}

hm_status check_dispatch(int64_t t, int32_t topk, int32_t num_experts) {
  if (t < 0 || topk < 1 || num_experts < 1 || num_experts > 512 || topk > num_experts) return HM_ERR_SHAPE;
  if (t > kMaxBlocks || t * (int64_t)topk >= (1ll << 31)) return HM_ERR_SHAPE;
  return HM_OK;
}

size_t dispatch_ws(int64_t t, int32_t topk, int32_t num_experts) {
  if (t * topk <= kSortDispatch) return 0;
  return (size_t)moe_sort_blocks(t * topk, nullptr) * (size_t)num_experts * sizeof(int32_t);
}

hm_status done(hipError_t e) { return e == hipSuccess ? HM_OK : HM_ERR_HIP; }

}  // namespace

HM_API hm_status hm_moe_dispatch_workspace_size(int64_t t, int32_t topk, int32_t num_experts, size_t* bytes) {
  if (!bytes) return HM_ERR_NULL;
  if (hm_status s = check_dispatch(t, topk, num_experts)) return s;
  *bytes = dispatch_ws(t, topk, num_experts);
  return HM_OK;
}

HM_API hm_status hm_moe_dispatch(const uint16_t* x, const int32_t* topk_ids, int64_t t, int32_t topk,
                                 int32_t num_experts, int64_t n, uint16_t* xs, int32_t* counts, int32_t* offsets,
                                 int32_t* sorted_pairs, int32_t* positions, void* ws, size_t ws_bytes,
                                 hipStream_t stream) {
  if (hm_status s = check_dispatch(t, topk, num_experts)) return s;
  if (hm_status s = check_rows(t, topk, n)) return s;
  if (t == 0) return HM_OK;
  if (!x || !topk_ids || !xs || !counts || !offsets || !sorted_pairs || !positions) return HM_ERR_NULL;
  if (!aligned(x, 16) || !aligned(xs, 16) || !aligned(topk_ids, 4) || !aligned(counts, 4) || !aligned(offsets, 4) ||
      !aligned(sorted_pairs, 4) || !aligned(positions, 4))
    return HM_ERR_ALIGN;
  const size_t need = dispatch_ws(t, topk, num_experts);
  if (need) {
    if (!ws) return HM_ERR_NULL;
    if (ws_bytes < need) return HM_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return HM_ERR_ALIGN;
  }
  if (t * topk <= kSmallPairs)
    return done(launch_dispatch_small(x, topk_ids, t, topk, num_experts, n, xs, counts, offsets, sorted_pairs, positions,
                                      stream));
  hipError_t e = t * topk <= kSortDispatch
                     ? launch_dispatch_sort(topk_ids, t * topk, num_experts, counts, offsets, sorted_pairs, positions,
                                            stream)
                     : launch_moe_sort_pos(topk_ids, t * topk, num_experts, counts, offsets, sorted_pairs, positions,
                                           static_cast<int32_t*>(ws), stream);
  if (e == hipSuccess) e = launch_dispatch_rows(x, positions, t, topk, n, xs, stream);
  return done(e);
}

HM_API hm_status hm_moe_dispatch_grad(const uint16_t* dxs, const int32_t* positions, int64_t t, int32_t topk,
                                      int64_t n, uint16_t* dx, hipStream_t stream) {
  if (hm_status s = check_rows(t, topk, n)) return s;
  if (t == 0) return HM_OK;
  if (!dxs || !positions || !dx) return HM_ERR_NULL;
  if (!aligned(dxs, 16) || !aligned(dx, 16) || !aligned(positions, 4)) return HM_ERR_ALIGN;
  return done(launch_collect(dxs, nullptr, positions, t, topk, n, dx, stream));
}

HM_API hm_status hm_moe_collect(const uint16_t* ys, const float* w, const int32_t* positions, int64_t t,
                                int32_t topk, int64_t n, uint16_t* out, hipStream_t stream) {
  if (hm_status s = check_rows(t, topk, n)) return s;
  if (t == 0) return HM_OK;
  if (!ys || !w || !positions || !out) return HM_ERR_NULL;
  if (!aligned(ys, 16) || !aligned(out, 16) || !aligned(w, 4) || !aligned(positions, 4)) return HM_ERR_ALIGN;
  return done(launch_collect(ys, w, positions, t, topk, n, out, stream));
}

HM_API hm_status hm_moe_collect_grad(const uint16_t* dout, const uint16_t* ys, const float* w,
                                     const int32_t* positions, int64_t t, int32_t topk, int64_t n, uint16_t* dys,
                                     float* dw, hipStream_t stream) {
  if (hm_status s = check_rows(t, topk, n)) return s;
  if (t == 0) return HM_OK;
  if (!dout || !ys || !w || !positions || !dys || !dw) return HM_ERR_NULL;
  if (!aligned(dout, 16) || !aligned(ys, 16) || !aligned(dys, 16) || !aligned(w, 4) || !aligned(positions, 4) ||
      !aligned(dw, 4))
    return HM_ERR_ALIGN;
  return done(launch_collect_grad(dout, ys, w, positions, t, topk, n, dys, dw, stream));
}
