"""The 8-bit integer layers at sizes that reach every kernel and way to cut the
work (the plan's text says which), against the definition in 64 bits on the GPU.

Bounds as in test_gpu_int8_layers: u = 2^-8 half a bf16 step, e = 2^-24 half an
fp32 step."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24
F = torch.float64


def _layer(seed, m, n, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = lambda r: (torch.randn(r, k, generator=g, device="cuda") * 40).round().clamp(-128, 127).to(torch.int8)     # noqa: E731
    s = lambda r, top: (torch.rand(r, generator=g, device="cuda") + 0.01) * top                                     # noqa: E731
    rows = lambda r, c: torch.randn(r, c, generator=g, device="cuda").to(torch.bfloat16)                            # noqa: E731
    return (q(m), s(m, 1 / 40), q(n), s(n, 1 / (40 * k ** 0.5))), rows


def _hats(a):
    return a[0].to(F) * a[1].to(F)[:, None], a[2].to(F) * a[3].to(F)[:, None]


def _product(a):
    """The whole-number sums (exact in fp64 in any order) times both scales."""
    return (a[0].to(F) @ a[2].to(F).t()) * a[1].to(F)[:, None] * a[3].to(F)


def _close(got, ref, lim, what):
    bad = ~((got.to(F) - ref).abs() <= lim)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), ref[bad][:3].tolist())


# every kernel for few rows: row blocks (of one group), weight blocks, one block or several to a compute unit
FEW = [
    (1, 4129, 128, "1 groups of 1 row blocks, weight blocks 1"), (1, 2, 384, "1 groups of 1 row blocks, weight blocks 1"),
    (11, 4222, 2560, "1 groups of 1 row blocks, weight blocks 2"), (43, 2093, 128, "2 groups of 2 row blocks, weight blocks 1"),
    (35, 1, 128, "2 groups of 2 row blocks, weight blocks 1"), (66, 12359, 128, "3 groups of 2 row blocks, weight blocks 2"),
    (19, 4131, 1920, "1 groups of 2 row blocks, weight blocks 2"), (196, 6275, 128, "7 groups of 2 row blocks, weight blocks 3"),
    (30, 8481, 2304, "1 groups of 2 row blocks, weight blocks 3"), (33, 4135, 128, "1 groups of 3 row blocks, weight blocks 1"),
    (33, 2082, 128, "1 groups of 3 row blocks, weight blocks 1"), (129, 6842, 128, "3 groups of 3 row blocks, weight blocks 2"),
    (46, 4097, 1024, "1 groups of 3 row blocks, weight blocks 2"), (169, 8255, 128, "4 groups of 3 row blocks, weight blocks 3"),
    (46, 8374, 1024, "1 groups of 3 row blocks, weight blocks 3"), (51, 10317, 128, "1 groups of 4 row blocks, weight blocks 1"),
    (49, 2094, 384, "1 groups of 4 row blocks, weight blocks 1"), (97, 10515, 128, "2 groups of 4 row blocks, weight blocks 2"),
    (59, 4237, 896, "1 groups of 4 row blocks, weight blocks 2"), (638, 2446, 640, "10 groups of 4 row blocks, weight blocks 3"),
    (115, 4107, 896, "2 groups of 4 row blocks, weight blocks 3"), (289, 5894, 128, "5 groups of 4 row blocks, weight blocks 4"),
    (294, 2831, 1664, "5 groups of 4 row blocks, weight blocks 4"), (65, 6873, 128, "1 groups of 5 row blocks, weight blocks 1"),
    (65, 2771, 256, "1 groups of 5 row blocks, weight blocks 1"), (65, 13037, 256, "1 groups of 5 row blocks, weight blocks 2"),
    (79, 4105, 768, "1 groups of 5 row blocks, weight blocks 2"), (147, 10159, 128, "2 groups of 5 row blocks, weight blocks 3"),
    (69, 8558, 896, "1 groups of 5 row blocks, weight blocks 3"), (129, 12314, 128, "2 groups of 5 row blocks, weight blocks 4"),
    (133, 6345, 1664, "2 groups of 5 row blocks, weight blocks 4"), (97, 6263, 256, "1 groups of 7 row blocks, weight blocks 1"),
    (97, 3105, 384, "1 groups of 7 row blocks, weight blocks 1"), (98, 12297, 128, "1 groups of 7 row blocks, weight blocks 2"),
    (101, 4103, 768, "1 groups of 7 row blocks, weight blocks 2"), (99, 8254, 640, "1 groups of 7 row blocks, weight blocks 3"),
    (202, 6265, 1408, "2 groups of 7 row blocks, weight blocks 4")]
FEW_GATED = [
    (1, 4117, 128, "1 groups of 1 row blocks, weight blocks 2"), (1, 1, 256, "1 groups of 1 row blocks, weight blocks 2"),
    (33, 2257, 128, "2 groups of 2 row blocks, weight blocks 2"), (65, 1, 128, "3 groups of 2 row blocks, weight blocks 2"),
    (34, 6413, 128, "1 groups of 3 row blocks, weight blocks 2"), (33, 2063, 256, "1 groups of 3 row blocks, weight blocks 2"),
    (49, 10251, 128, "1 groups of 4 row blocks, weight blocks 2"), (49, 2171, 384, "1 groups of 4 row blocks, weight blocks 2"),
    (50, 12461, 128, "1 groups of 4 row blocks, weight blocks 4"), (51, 4157, 2048, "1 groups of 4 row blocks, weight blocks 4"),
    (65, 4237, 384, "1 groups of 5 row blocks, weight blocks 2"), (68, 2727, 384, "1 groups of 5 row blocks, weight blocks 2"),
    (65, 10766, 128, "1 groups of 5 row blocks, weight blocks 4"), (75, 4137, 1664, "1 groups of 5 row blocks, weight blocks 4"),
    (194, 3075, 128, "2 groups of 7 row blocks, weight blocks 2"), (97, 2275, 512, "1 groups of 7 row blocks, weight blocks 2"),
    (204, 2185, 1408, "2 groups of 7 row blocks, weight blocks 4")]
FORWARD = FEW + [
    (1030, 700, 128, "at once: 54 whole, 0 in 1"), (1232, 101, 640, "128x128: 10 whole"), (1050, 600, 4096, "0 whole, 45 in 4"),
    (1021, 4099, 7168, "256 whole, 8 in"), (1100, 300, 8320, "0 whole, 27 in 5"), (1025, 1300, 128, "at once: 99 whole"),
    (2000, 5201, 256, "at once: 656"), (2049, 7169, 2176, "at once: 969 whole"), (3528, 4489, 640, "256x256: 252"),
    (4090, 8101, 1152, "256x256: 512"), (4097, 5000, 128, "at once: 1320")]


@pytest.mark.parametrize("m,n,k,plan", FORWARD)
def test_product(m, n, k, plan):
    import quantized_gemm_int4_amd as hm
    assert plan in hm.hm_gemm_int8_plan(hm.HM_INT8_GEMM, m, n, k)
    a, _ = _layer(m + n + k, m, n, k)
    ref = _product(a)
    y = torch.full((m + 1, n), 7.0, dtype=torch.bfloat16, device="cuda")
    hm.hm_gemm_int8(*a, y=y[:m])
    _close(y[:m], ref, ref.abs() * (U + 4 * E), "y")
    assert bool((y[m] == 7).all())
    again = hm.hm_gemm_int8(*a)
    assert torch.equal(again, y[:m])


GATED = FEW_GATED + [
         (1030, 350, 128, "at once: 54 whole, 0 in 1"), (1232, 101, 640, "128x128: 20 whole"), (1050, 300, 4096, "0 whole, 45 in 4"),
         (1021, 2049, 7168, "256 whole, 8 in"), (2000, 2601, 256, "at once: 656"), (3528, 2245, 1664, "256x256: 252"),
         (4090, 4001, 2304, "256x256: 512")]


@pytest.mark.parametrize("m,d,k,plan", GATED)
def test_gated_and_its_gradient(m, d, k, plan):
    import quantized_gemm_int4_amd as hm
    assert plan in hm.hm_gemm_int8_plan(hm.HM_INT8_GATED, m, 2 * d, k)
    assert plan in hm.hm_gemm_int8_plan(hm.HM_INT8_GATED_GRAD, m, 2 * d, k)
    a, rows = _layer(m + d + k, m, 2 * d, k)
    g, u = _product(a).chunk(2, 1)
    s, rest = torch.sigmoid(g), torch.sigmoid(-g)
    c = (60 + 4 * g.abs()) * 2 * E
    h = torch.full((m + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    hm.hm_gemm_int8_gated(*a, h=h[:m])
    ref = g * s * u
    _close(h[:m], ref, ref.abs() * (U + c) + 1e-30, "h")
    dh = rows(m, d)
    out = torch.full((m + 1, 2 * d), 7.0, dtype=torch.bfloat16, device="cuda")
    hm.hm_gemm_int8_gated_grad(dh, *a, dgu=out[:m])
    f = dh.to(F)
    du, dg = f * g * s, f * u * s * (1 + g * rest)
    _close(out[:m, d:], du, du.abs() * (U + c) + 1e-30, "du")
    _close(out[:m, :d], dg, dg.abs() * U + (f * u).abs() * s * (1 + g.abs() * rest) * 2 * c + 1e-30, "dg")
    assert bool((h[m] == 7).all()) and bool((out[m] == 7).all())


GRAD = [(100, 300, 256, "few rows: groups of 32", "of codes"), (1, 7, 128, "few rows: groups of 32", "of codes, two at once: 1 whole"),
        (1100, 4096, 384, "few rows: groups of 32", "of codes"), (333, 7168, 2048, "few rows: groups of 64", "of codes, two at once: 896"),
        (244, 2065, 3840, "few rows: groups of 64", "of codes"), (851, 3968, 1792, "few rows: groups of 128", "of codes, two at once"),
        (646, 6806, 2048, "few rows: groups of 128", "256x256: 216"), (131, 2584, 1408, "few rows: groups of 32", "of codes: 231 whole"),
        (64, 14336, 1024, "of codes: 0 whole, 8 in", "dw"), (1315, 1, 128, "few rows", "of codes: 0 whole, 1 in 4"),
        (2121, 1, 128, "of codes, two at once: 17 whole", "of codes: 0 whole, 1 in"), (1368, 129, 2688, "of codes: 231 whole", "of codes: 42 whole"),
        (1500, 6000, 2048, "128x128: 192 whole", "dw"), (3000, 5003, 1024, "128x128: 192 whole", "128x128, two at once: 320 whole"),
        (4096, 4100, 1152, "128x128: 256 whole, 32 in", "128x128: 256 whole, 41 in"), (2828, 3620, 384, "of codes: 0 whole, 69 in", "128x128: 87 whole"),
        (5100, 4100, 4096, "128x128, two at once: 1280", "128x128: 1024 whole, 32 in"), (2600, 2600, 4096, "256x256: 176", "256x256: 176"),
        (5100, 4100, 6016, "256x256: 480", "256x256: 408")]


@pytest.mark.parametrize("m,n,k,dxp,dwp", GRAD)
def test_gradient(m, n, k, dxp, dwp):
    import quantized_gemm_int4_amd as hm
    one, two = hm.hm_gemm_int8_plan(hm.HM_INT8_GRAD, m, n, k).split("; ")
    assert dxp in one and dwp in two, (one, two)
    a, rows = _layer(m + n + k, m, n, k)
    x, w = _hats(a)
    dy = rows(m, n) * 0.05
    f = dy.to(F)
    dx = torch.full((m + 1, k), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((n + 1, k), 7.0, dtype=torch.bfloat16, device="cuda")
    hm.hm_gemm_int8_grad(dy, *a, dx=dx[:m], dw=dw[:n])
    for name, got, ref, b, terms in (("dx", dx[:m], f @ w, f.abs() @ w.abs(), n), ("dw", dw[:n], f.t() @ x, f.abs().t() @ x.abs(), m)):
        _close(got, ref, b * (U + (terms + 2) * 2 * E) * (1 + U) + ref.abs() * U + 1e-30, name)
        # two independent roundings of at most u, see test_gpu_int8_layers
        assert float((got.to(F) - ref).norm() / ref.norm()) <= U, name
    assert bool((dx[m] == 7).all()) and bool((dw[n] == 7).all())
    # one of the two alone, and again: the same bits
    one, _ = hm.hm_gemm_int8_grad(dy, *a, need_dw=False)
    _, two = hm.hm_gemm_int8_grad(dy, *a, need_dx=False)
    assert torch.equal(one, dx[:m]) and torch.equal(two, dw[:n])


@pytest.mark.parametrize("m,n,k", [g[:3] for g in GRAD if g[0] > 2])
def test_an_infinity_at_the_start_of_a_row_stays_in_it(m, n, k):
    """Behind the end of the row before it: the tile of that row must not see it."""
    import quantized_gemm_int4_amd as hm
    a, rows = _layer(m + n + k, m, n, k)
    dy = rows(m, n)
    dy[1, 0] = float("inf")
    dx, dw = hm.hm_gemm_int8_grad(dy, *a)
    dx, dw = dx.isfinite().all(1), dw.isfinite().all(1)
    assert int((~dx).sum()) == 1 and not bool(dx[1]), (~dx).nonzero()[:5]
    assert int((~dw).sum()) == 1 and not bool(dw[0]), (~dw).nonzero()[:5]



def test_gradient_against_differences():
    """A loss of the product along random directions of x_hat and w_hat: its
    central difference is the gradient's inner product with the direction (the
    loss is quadratic, so the difference has no error of its own)."""
    import quantized_gemm_int4_amd as hm
    m, n, k = 300, 520, 384
    a, rows = _layer(5, m, n, k)
    x, w = _hats(a)
    dy = rows(m, n)
    dx, dw = hm.hm_gemm_int8_grad(dy, *a)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    vx, vw = torch.randn(m, k, generator=g, device="cuda", dtype=F), torch.randn(n, k, generator=g, device="cuda", dtype=F)
    loss = lambda p, q: float((dy.to(F) * (p @ q.t())).sum())                                   # noqa: E731
    for got, v, diff in ((dx, vx, loss(x + vx, w) - loss(x - vx, w)), (dw, vw, loss(x, w + vw) - loss(x, w - vw))):
        # every element of the gradient is off by at most 2 u (1 + u) of its terms' absolute sum, which its own
        # rounding noise stays under by the square root of their number; bounded here by the sum over all elements
        inner = float((got.to(F) * v).sum())
        size = float((got.to(F).abs() * v.abs()).sum())
        assert abs(inner - diff / 2) <= 2 * U * size, (inner, diff / 2, size)


def test_adapters_beside_an_int8_layer():
    """An adapter trained on a layer whose weights stay in 8 bits: the layer's
    product is the adapters' base, its gradient their dx_base."""
    import quantized_gemm_int4_amd as hm
    m, n, k, rank, L = 130, 260, 384, 16, 3
    a, rows = _layer(9, m, n, k)
    x = (a[0].float() * a[1][:, None]).to(torch.bfloat16)
    ids = (torch.arange(m, device="cuda") % (L + 1) - 1).to(torch.int32)
    A, B = rows(L, rank * k).view(L, rank, k) * k ** -0.5, rows(L, n * rank).view(L, n, rank) * 0.1
    A, B, sc = A.contiguous(), B.contiguous(), torch.ones(L, device="cuda")
    d, h = hm.lora_desc(n, k, rank, L), torch.empty(m, rank, device="cuda")
    base = hm.hm_gemm_int8(*a)
    y = hm.hm_lora(d, x, ids, A, B, sc, base=base, h=h)
    dy = rows(m, n)
    dxb, _ = hm.hm_gemm_int8_grad(dy, *a, need_dw=False)
    dx, da, db = hm.hm_lora_grad(d, dy, x, h, ids, A, B, sc, dx_base=dxb)
    yr, dxr = base.to(F), dxb.to(F)
    for e in range(L):
        r = (ids == e).nonzero()[:, 0]
        yr[r] += x[r].to(F) @ A[e].to(F).t() @ B[e].to(F).t()
        dxr[r] += dy[r].to(F) @ B[e].to(F) @ A[e].to(F)
    # sums of a few hundred terms in fp32, one rounding: 2 u of the result and its base cover both
    assert bool(((y.to(F) - yr).abs() <= U * yr.abs() + 2.0 ** -12 * (yr.abs() + base.to(F).abs() + 1)).all())
    assert bool(((dx.to(F) - dxr).abs() <= U * dxr.abs() + 2.0 ** -12 * (dxr.abs() + dxb.to(F).abs() + 1)).all())
