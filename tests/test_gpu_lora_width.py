"""The width in which h and g enter the adapters' second products: all 24 bits
of the fp32 values.  A sum that cancels all but the last eight of 18
significant bits shows what a narrower operand would drop."""
import numpy as np
import pytest
import torch

from gpu_util import to_dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -8                 # half a bf16 step relative to the value

# m, n, k, rank, adapters: one-launch calls, calls without a grouping launch, units of 16, 32 and 64 rows
SHAPES = [(1, 40, 128, 8, 1), (5, 40, 256, 24, 2), (12, 70, 128, 64, 2), (12, 70, 128, 128, 2), (50, 40, 128, 16, 2),
          (50, 300, 256, 64, 3), (100, 40, 128, 16, 20), (150, 136, 256, 32, 6), (120, 72, 128, 128, 5),
          (300, 264, 256, 48, 2), (300, 72, 128, 128, 2), (700, 300, 256, 16, 1), (1400, 40, 128, 64, 1)]

# v and w are fp32 values that differ in v's last eight significant bits of 18; every result below is v - w, and what a
# narrower operand drops is all of it.  At most eight additions of values below 2.01 touch a result: 2^-23 each of 2.01.
TAIL = 2.0 ** -17
WIDTH_ERR = 8 * 2.01 * 2.0 ** -23 + U * TAIL


@pytest.mark.parametrize("m,n,k,rank,L", SHAPES)
def test_h_and_g_enter_the_products_in_full_width(m, n, k, rank, L):
    import quantized_gemm_int4_amd as hm
    d, bf, r = hm.lora_desc(n, k, rank, L), torch.bfloat16, np.random.default_rng(m)
    z = lambda *s: torch.zeros(*s, dtype=bf, device="cuda")                               # noqa: E731
    one = torch.ones(L, device="cuda")
    ids = r.integers(0, L, m).astype(np.int32)
    idt = to_dev(ids)
    tail = torch.tensor([1.0, 2.0 ** -9, 2.0 ** -17], device="cuda").to(bf)
    even = torch.arange(0, rank, 2, device="cuda")

    def pairs(count):
        """[count, rank]: +1 and -1 at one pair of ranks per row"""
        p = z(count, rank)
        i = 2 * (torch.arange(count, device="cuda") % (rank // 2))
        p.scatter_(1, i[:, None], torch.ones(count, 1, dtype=bf, device="cuda"))
        p.scatter_(1, i[:, None] + 1, -torch.ones(count, 1, dtype=bf, device="cuda"))
        return p

    # forward: h = v at even ranks, w at odd ones; y = v - w
    x, a = z(m, k), z(L, rank, k)
    x[:, :3] = tail
    a[:, :, :3] = 1
    a[:, even + 1, 2] = 0
    b = pairs(n).expand(L, n, rank).contiguous()
    y = hm.hm_lora(d, x, idt, a, b, one)
    assert ((y.double() - TAIL).abs() <= WIDTH_ERR).all()

    # dx: g = v at even ranks, w at odd ones
    dy, b = z(m, n), z(L, n, rank)
    dy[:, :3] = 1
    b[:, :3] = tail[:, None]
    b[:, 2, even + 1] = 0
    a = pairs(k).t().expand(L, rank, k).contiguous()
    h = torch.zeros(m, rank, device="cuda")
    dx, _, _ = hm.hm_lora_grad(d, dy, x, h, idt, a, b, one)
    assert ((dx.double() - TAIL).abs() <= WIDTH_ERR).all()

    # da, db: two rows of an adapter, v and w, with opposite signs in x and dy
    two = [np.nonzero(ids == e)[0] for e in range(L)]
    two = [(e, int(v[0]), int(v[-1])) for e, v in enumerate(two) if len(v) > 1]
    x, dy, b = z(m, k), z(m, n), z(L, n, rank)
    b[:, :3] = tail[:, None]
    for _, p, q in two:
        x[p], x[q] = 1, -1
        dy[p, :3] = 1
        dy[q, :2] = 1
    _, da, _ = hm.hm_lora_grad(d, dy, x, h, idt, a, b, one, need_dx=False)
    dy = z(m, n)
    for _, p, q in two:
        h[p], h[q] = 1 + 2.0 ** -9 + TAIL, 1 + 2.0 ** -9
        dy[p], dy[q] = 1, -1
    _, _, db = hm.hm_lora_grad(d, dy, x, h, idt, a, b, one, need_dx=False)
    for e, _, _ in two:
        assert ((da[e].double() - TAIL).abs() <= WIDTH_ERR).all() and ((db[e].double() - TAIL).abs() <= WIDTH_ERR).all()
