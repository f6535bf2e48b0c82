"""The collect's gradient of more than 2^23 tokens, with rows longer than 2048:
sampled tokens against fp64 products (34 GB an array)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_collect_gradient_past_2_23_tokens():
    import quantized_gemm_int4_amd as hm
    t, n, bf = (1 << 23) + 5, 2056, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(2)
    dout, ys = (torch.empty(t, n, dtype=bf, device="cuda").normal_(generator=g) for _ in range(2))
    w = torch.rand(t, 1, generator=g, device="cuda")
    pos = torch.arange(t, device="cuda", dtype=torch.int32).flip(0).reshape(t, 1).contiguous()
    pick = torch.cat([torch.arange(64), torch.randint(0, t, (256,)), torch.arange(t - 64, t)]).cuda()
    rows = ys[pos[pick, 0].long()].clone()
    dys, dw = hm.hm_moe_collect_grad(dout, ys, w, pos, dys=ys)
    d = dout[pick]
    want = d.float() * w[pick]                                  # one fp32 rounding, then bf16's
    assert torch.equal(dys[pos[pick, 0].long()], want.to(bf))
    p = d.double() * rows.double()
    # n products summed in fp32, each addition off by at most 2^-24 of the sum of absolute terms, taken twice
    assert ((dw[pick, 0].double() - p.sum(1)).abs() <= (n + 8) * 2.0 ** -23 * p.abs().sum(1)).all()
    del dout, ys, dys
    torch.cuda.empty_cache()
