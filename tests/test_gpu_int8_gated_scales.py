"""Scales that are not finite in the gated block of the 8-bit integer layers and its
gradient, on every kernel: a token's spoils its row, a gate channel's its column of h,
dg and du, an up channel's its column of h and dg only (du does not depend on the up
product), and nothing else.  The rest has the bits of the same call with finite scales."""
import pytest
import torch

pytestmark = pytest.mark.gpu

# few rows, 128 x 128 tiles with the last ones cut, two blocks a unit, 256 x 256 tiles
SIZES = [(5, 300, 256, "few"), (70, 257, 128, "few"), (1050, 300, 4096, "0 whole, 45 in"), (1030, 350, 128, "at once"),
         (1232, 101, 640, "128x128: 20 whole"), (3528, 2245, 1664, "256x256")]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("m,d,k,plan", SIZES)
def test_they_stay_in_their_row_and_column(m, d, k, plan, bad):
    import quantized_gemm_int4_amd as hm
    assert plan in hm.hm_gemm_int8_plan(hm.HM_INT8_GATED, m, 2 * d, k)
    assert plan in hm.hm_gemm_int8_plan(hm.HM_INT8_GATED_GRAD, m, 2 * d, k)
    g = torch.Generator(device="cuda")
    g.manual_seed(m + d + k)
    one = dict(generator=g, device="cuda")
    q = lambda r: torch.randint(-128, 128, (r, k), dtype=torch.int8, **one)                     # noqa: E731
    x8, w8 = q(m), q(2 * d)
    sx, sw = (torch.rand(m, **one) + 0.5) / 128, (torch.rand(2 * d, **one) + 0.5) / (64 * k ** 0.5)
    dh = torch.randn(m, d, **one).to(torch.bfloat16)
    h, dgu = hm.hm_gemm_int8_gated(x8, sx, w8, sw), hm.hm_gemm_int8_gated_grad(dh, x8, sx, w8, sw)
    assert bool(h.isfinite().all()) and bool(dgu.isfinite().all())
    row, gates, ups = m - 1, [7, d - 1], [0, 65]               # at the ends and within
    sx[row] = bad
    sw[gates] = bad
    sw[[d + c for c in ups]] = bad
    h2, dgu2 = hm.hm_gemm_int8_gated(x8, sx, w8, sw), hm.hm_gemm_int8_gated_grad(dh, x8, sx, w8, sw)
    for name, got, ref, cols in (("h", h2, h, gates + ups), ("dg", dgu2[:, :d], dgu[:, :d], gates + ups), ("du", dgu2[:, d:], dgu[:, d:], gates)):
        hit = torch.zeros(m, d, dtype=torch.bool, device="cuda")
        hit[row], hit[:, cols] = True, True
        assert not bool(got[hit].isfinite().any()), (name, "finite where it should not be", (got.isfinite() & hit).nonzero()[:5].tolist())
        assert torch.equal(got[~hit], ref[~hit]), name
