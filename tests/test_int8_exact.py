"""The gradients' exact inputs on the CPU: their conditions hold, any order of summation
gives the same bits, and small mistakes planted in the reference show."""
import pytest
import torch

import int8_exact as ex

SIZES = [(333, 7168, 128), (70, 100, 128), (1500, 600, 256), (1, 7, 128), (2121, 1, 128)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_sums_are_exact_in_any_order(m, n, k):
    dy, a = ex.whole(m, n, k, "cpu", m + n)
    x, w = ex.operand(a[0], a[1]), ex.operand(a[2], a[3])
    assert torch.equal(w.double(), a[2].double() * a[3].double()[:, None])       # (powers of two: nothing is rounded)
    for f, o, terms in ((dy, w, n), (dy.t(), x, m)):
        assert float((f.double().abs() @ o.double().abs()).max()) * 2 <= 2 ** 24
        ref = f.double() @ o.double()
        p = torch.randperm(terms, generator=torch.Generator().manual_seed(1))
        some = torch.zeros(f.shape[0], k)
        for lo in range(0, terms, 97):                         # fp32 sums of another order
            some += f[:, p[lo:lo + 97]].float() @ o[p[lo:lo + 97]].float()
        assert torch.equal(some.double(), ref)


@pytest.mark.parametrize("m,n,k", SIZES[:3])
def test_planted_mistakes_show(m, n, k):
    dy, a = ex.whole(m, n, k, "cpu", m + n)
    every = slice(None)
    dx, dw = ex.whole_results(dy, a, every, every)
    # the last row of the contraction lost in one 32 x 32 block of results
    for ref, f, o in ((dx, dy, ex.operand(a[2], a[3])), (dw, dy.t(), ex.operand(a[0], a[1]))):
        lost = f[:32, -1:].double() @ o[-1:, :32].double()
        got = ((f[:32].double() @ o[:, :32].double()) - lost).float().to(torch.bfloat16)
        assert int((got != ref[:32, :32]).sum()) > 100
    # every channel with its neighbour's scale
    wrong = (a[0], a[1].roll(1), a[2], a[3].roll(1))
    dx2, dw2 = ex.whole_results(dy, wrong, every, every)
    assert not torch.equal(dx2, dx) and not torch.equal(dw2, dw)
    # an operand that is not rounded, or rounded towards zero
    (dyx, col, vx), _, b = ex.chosen(m, n, k, "cpu", m)
    ref = ex.chosen_result(col, vx, b[2], b[3])
    exact = b[2][col].double() * b[3][col].double()[:, None]
    cut = ((b[2][col].float() * b[3][col][:, None]).view(torch.int32) & -65536).view(torch.float32)
    for o in (exact, cut):
        assert int(((vx.double()[:, None] * o.double()).to(torch.bfloat16) != ref).sum()) > ref.numel() // 20


@pytest.mark.parametrize("m,n,k", SIZES)
def test_chosen_terms_are_the_definition(m, n, k):
    (dyx, col, vx), (dyw, row, vw), a = ex.chosen(m, n, k, "cpu", m)
    dx = dyx.double() @ ex.operand(a[2], a[3]).double()
    dw = dyw.t().double() @ ex.operand(a[0], a[1]).double()
    assert torch.equal(ex.chosen_result(col, vx, a[2], a[3]), dx.float().to(torch.bfloat16))
    assert torch.equal(ex.chosen_result(row, vw, a[0], a[1]), dw.float().to(torch.bfloat16))
