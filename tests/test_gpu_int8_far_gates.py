"""Gates far below zero in the gated block of the 8-bit integer layers: silu(g) and
its derivative are then under fp32's normal range (below g = -87) or under its
smallest number (below -104), but their products with a large up value or
gradient are not.  Against the definition in 64 bits, on every kernel.

Bounds as in test_gpu_int8_layers: u = 2^-8 half a bf16 step, e = 2^-24 half an fp32 step; g and u are off by 3 e
each, the relative condition of silu and of its derivative is at most 1 + |g|, the exponential and the
reciprocal are off by (48 + |g|) 2 e, together (60 + 4 |g|) 2 e.  Results under 2^-126 may lose all bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U, E, TINY = 2.0 ** -8, 2.0 ** -24, 2.0 ** -126
F = torch.float64

# few rows, 128 x 128 tiles with the last ones cut, two blocks a unit, 256 x 256 tiles
SIZES = [(1, 300, 128, "few"), (37, 257, 256, "few"), (1050, 300, 4096, "0 whole, 45 in"), (1030, 350, 128, "at once"),
         (1232, 101, 640, "128x128: 20 whole"), (3528, 2245, 1664, "256x256")]


def _close(got, ref, lim, what):
    bad = ~((got.to(F) - ref).abs() <= lim)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), ref[bad][:3].tolist())


def _far(m, d, k):
    """A layer with gates from -64 to -178 and up values to 2^88; gate, up in 64 bits, and their bound."""
    g = torch.Generator(device="cuda")
    g.manual_seed(m + d + k)
    one = dict(generator=g, device="cuda")
    x8, w8 = torch.zeros(m, k, dtype=torch.int8, device="cuda"), torch.zeros(2 * d, k, dtype=torch.int8, device="cuda")
    last = k - 1                                               # the one term of every sum: in the last part of a cut tile
    x8[:, last] = 1
    w8[:d, last] = -(64 + torch.arange(d, device="cuda") % 64).to(torch.int8)
    w8[d:, last] = torch.randint(1, 128, (d,), **one).to(torch.int8)
    sx = torch.where(torch.arange(m, device="cuda") % 2 == 0, 1.0, 1.4)
    sw = torch.cat([torch.ones(d, device="cuda"), torch.exp2(torch.randint(0, 81, (d,), **one).float())])
    gate, up = ((x8[:, last:].to(F) @ w8[:, last:].to(F).t()) * sx.to(F)[:, None] * sw.to(F)).chunk(2, 1)
    return (x8, sx, w8, sw), gate, up, (60 + 4 * gate.abs()) * 2 * E, one


@pytest.mark.parametrize("m,d,k,plan", SIZES)
def test_gradient(m, d, k, plan):
    """dh to 2^32 (dh u stays under 2^121)."""
    import quantized_gemm_int4_amd as hm
    assert plan in hm.hm_gemm_int8_plan(hm.HM_INT8_GATED_GRAD, m, 2 * d, k)
    a, gate, up, c, one = _far(m, d, k)
    dh = (torch.randn(m, d, **one) * torch.exp2(torch.randint(0, 31, (m, d), **one).float())).to(torch.bfloat16)
    s, rest, f = torch.sigmoid(gate), torch.sigmoid(-gate), dh.to(F)
    dgu = hm.hm_gemm_int8_gated_grad(dh, *a)
    du, dg = f * gate * s, f * up * s * (1 + gate * rest)
    _close(dgu[:, d:], du, du.abs() * (U + c) + TINY, "du")
    _close(dgu[:, :d], dg, dg.abs() * U + (f * up).abs() * s * (1 + gate.abs() * rest) * 2 * c + TINY, "dg")


@pytest.mark.parametrize("m,d,k,plan", SIZES)
def test_forward(m, d, k, plan):
    import quantized_gemm_int4_amd as hm
    assert plan in hm.hm_gemm_int8_plan(hm.HM_INT8_GATED, m, 2 * d, k)
    a, gate, up, c, _ = _far(m, d, k)
    ref = gate * torch.sigmoid(gate) * up
    _close(hm.hm_gemm_int8_gated(*a), ref, ref.abs() * (U + c) + TINY, "h")


@pytest.mark.parametrize("m,d,k,plan", SIZES)
def test_largest_values(m, d, k, plan):
    """Up values, gradients and their products next to fp32's largest number, against gates from -80 on: no
    intermediate result may pass it."""
    import quantized_gemm_int4_amd as hm
    assert plan in hm.hm_gemm_int8_plan(hm.HM_INT8_GATED, m, 2 * d, k)
    x8, w8 = torch.zeros(m, k, dtype=torch.int8, device="cuda"), torch.zeros(2 * d, k, dtype=torch.int8, device="cuda")
    x8[:, 0] = 1
    w8[:d, 0] = -(80 + torch.arange(d, device="cuda") % 48).to(torch.int8)
    w8[d:, 0] = 127
    sx = torch.ones(m, device="cuda")
    gate = w8[:d, 0].to(F)[None].expand(m, d)
    s, c = torch.sigmoid(gate), (60 + 4 * gate.abs()) * 2 * E
    for up, grad in ((2.0 ** 120, 1.0), (127.0 ** -1, 2.0 ** 127), (2.0 ** 60, 2.0 ** 60)):  # up values of 127 times that
        a = (x8, sx, w8, torch.cat([torch.ones(d, device="cuda"), torch.full((d,), up, device="cuda")]))
        dh = torch.full((m, d), grad, dtype=torch.bfloat16, device="cuda")
        u = 127.0 * float(torch.tensor(up, dtype=torch.float32))
        ref = gate * s * u
        _close(hm.hm_gemm_int8_gated(*a), ref, ref.abs() * (U + c) + TINY, ("h", up))
        dgu = hm.hm_gemm_int8_gated_grad(dh, *a)
        du, dg = grad * gate * s, grad * u * s * (1 + gate * torch.sigmoid(-gate))
        _close(dgu[:, d:], du, du.abs() * (U + c) + TINY, ("du", grad))
        _close(dgu[:, :d], dg, dg.abs() * U + (grad * u * s * (1 + gate.abs())) * 2 * c + TINY, ("dg", up, grad))
