"""The 8-bit integer layers on arrays beyond 4 GiB, where offsets leave 32 bits:
rows from the start, the middle and the end against the definition in 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24
F = torch.float64


def _codes(r, k, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-128, 128, (r, k), generator=g, device="cuda", dtype=torch.int8)


def _some(m):
    return torch.tensor([0, 1, m // 2, m - 300, m - 2, m - 1], device="cuda")


@pytest.mark.parametrize("m,n,k", [(40000, 100, 130944), (50, 40000, 130944), (300000, 8192, 128), (64, 4194303, 1152)])
def test_product(m, n, k):
    """x8 of 5.2 GB, w8 of 5.2 GB, y of 4.9 GB, w8 of 4.8 GB."""
    import quantized_gemm_int4_amd as hm
    a = (_codes(m, k, 1), torch.rand(m, device="cuda") + 0.1, _codes(n, k, 2), torch.rand(n, device="cuda") / k)
    y = hm.hm_gemm_int8(*a)
    r = _some(m) if m > 300 else torch.arange(m, device="cuda")
    c = _some(n) if n > 10000 else torch.arange(n, device="cuda")
    ref = (a[0][r].to(F) @ a[2][c].to(F).t()) * a[1][r].to(F)[:, None] * a[3][c].to(F)
    lim = ref.abs() * (U + 4 * E)
    assert bool(((y[r][:, c].to(F) - ref).abs() <= lim).all())


@pytest.mark.parametrize("m,d,k", [(300000, 4096, 128), (100, 20000, 130944)])
def test_gated_and_its_gradient(m, d, k):
    """dgu of 4.9 GB; gate and up rows of 2.6 GB each."""
    import quantized_gemm_int4_amd as hm
    a = (_codes(m, k, 3), (torch.rand(m, device="cuda") + 0.1) / k, _codes(2 * d, k, 4), torch.rand(2 * d, device="cuda") / 64)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    dh = torch.randn(m, d, generator=g, device="cuda", dtype=torch.bfloat16)
    h, dgu = hm.hm_gemm_int8_gated(*a), hm.hm_gemm_int8_gated_grad(dh, *a)
    r = _some(m) if m > 300 else torch.arange(m, device="cuda")
    c = _some(d)
    p = lambda c: (a[0][r].to(F) @ a[2][c].to(F).t()) * a[1][r].to(F)[:, None] * a[3][c].to(F)   # noqa: E731
    gate, up, f = p(c), p(c + d), dh[r][:, c].to(F)
    s, rest = torch.sigmoid(gate), torch.sigmoid(-gate)
    e = (60 + 4 * gate.abs()) * 2 * E
    for got, ref, lim in ((h[r][:, c], gate * s * up, (gate * s * up).abs() * (U + e)),
                          (dgu[r][:, c + d], f * gate * s, (f * gate * s).abs() * (U + e)),
                          (dgu[r][:, c], f * up * s * (1 + gate * rest), (f * up).abs() * s * (1 + gate.abs() * rest) * (U + 2 * e))):
        assert bool(((got.to(F) - ref).abs() <= lim + 1e-30).all())


@pytest.mark.parametrize("m,n,k", [(300000, 8192, 128), (20000, 120000, 128), (40, 40000, 130944)])
def test_gradient(m, n, k):
    """dy of 4.9 and 4.8 GB, weights of 5.2 GB."""
    import quantized_gemm_int4_amd as hm
    a = (_codes(m, k, 6), (torch.rand(m, device="cuda") + 0.1) / 64, _codes(n, k, 7), (torch.rand(n, device="cuda") + 0.1) / 64)
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    dy = torch.randn(m, n, generator=g, device="cuda", dtype=torch.bfloat16)
    dx, dw = hm.hm_gemm_int8_grad(dy, *a)
    r, c = _some(m) if m > 300 else torch.arange(m, device="cuda"), _some(n)
    w, x = a[2].to(F) * a[3].to(F)[:, None], a[0].to(F) * a[1].to(F)[:, None]
    f = dy[r].to(F)
    for got, ref, b, terms in ((dx[r], f @ w, f.abs() @ w.abs(), n),
                               (dw[c], dy[:, c].to(F).t() @ x, dy[:, c].to(F).abs().t() @ x.abs(), m)):
        # fp32 sums: runs of 64 terms in the matrix cores' own sums, then one addition a run: terms / 64 + 64 roundings
        assert bool(((got.to(F) - ref).abs() <= b * (U + terms * 2 * E) * (1 + U) + ref.abs() * U).all())
        assert float((got.to(F) - ref).norm() / ref.norm()) <= U


def test_rows():
    """6.4 GB of rows: codes and scales at both ends."""
    import quantized_gemm_int4_amd as hm
    m, k = 200000, 16000
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x = torch.randn(m, k, generator=g, device="cuda", dtype=torch.bfloat16)
    q, s = hm.hm_quant_int8_rows(x)
    r = _some(m)
    amax = x[r].abs().amax(1, keepdim=True).to(F)
    assert torch.equal(q[r].to(F), torch.round(x[r].to(F) * 127 / amax))
    assert torch.equal(s[r], amax[:, 0].float() / 127)
