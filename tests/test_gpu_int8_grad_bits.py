"""The gradients of the 8-bit integer layers bit by bit, at sizes that reach every kernel
and way to cut the work and on arrays beyond 4 GiB: inputs whose sums are exact in any
order, and single terms, which show the operand's rounding (int8_exact)."""
import pytest
import torch

import int8_exact as ex
from test_gpu_int8_paths import GRAD

pytestmark = pytest.mark.gpu
SIZES = [g[:3] for g in GRAD] + [(5, 3, 128), (64, 64, 128), (65, 130, 256), (127, 257, 384), (129, 33, 1152), (300, 515, 896)]


def _same(got, ref, what):
    bad = got != ref
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), ref[bad][:3].tolist())


@pytest.mark.parametrize("m,n,k", SIZES)
def test_exact_sums(m, n, k):
    import quantized_gemm_int4_amd as hm
    dy, a = ex.whole(m, n, k, "cuda", m + n + k)
    dx, dw = hm.hm_gemm_int8_grad(dy, *a)
    for name, got, ref in zip(("dx", "dw"), (dx, dw), ex.whole_results(dy, a, slice(None), slice(None))):
        _same(got, ref, name)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_single_terms(m, n, k):
    import quantized_gemm_int4_amd as hm
    (dyx, col, vx), (dyw, row, vw), a = ex.chosen(m, n, k, "cuda", m + n + k)
    dx, _ = hm.hm_gemm_int8_grad(dyx, *a, need_dw=False)
    _same(dx, ex.chosen_result(col, vx, a[2], a[3]), "dx")
    _, dw = hm.hm_gemm_int8_grad(dyw, *a, need_dx=False)
    _same(dw, ex.chosen_result(row, vw, a[0], a[1]), "dw")


@pytest.mark.parametrize("m,n,k", [(300000, 8192, 128), (20000, 120000, 128), (40, 40000, 130944)])
def test_exact_sums_beyond_4_gib(m, n, k):
    """dy of 4.9 and 4.8 GB, weights of 5.2 GB: results from the start, the middle and the end."""
    import quantized_gemm_int4_amd as hm
    dy, a = ex.whole(m, n, k, "cuda", 11)
    dx, dw = hm.hm_gemm_int8_grad(dy, *a)
    some = lambda r: torch.arange(r, device="cuda") if r <= 300 else torch.tensor([0, 1, r // 2, r - 300, r - 2, r - 1], device="cuda")  # noqa: E731
    rows, cols = some(m), some(n)
    for name, got, ref in zip(("dx", "dw"), (dx[rows], dw[cols]), ex.whole_results(dy, a, rows, cols)):
        _same(got, ref, name)
