"""The gradient of hm_moe_combine: hm_moe_collect_grad with each pair's own row
as its position.  Both sides of the combine against the oracle, and the
collect with those positions gives the combine's bits."""
import numpy as np
import pytest
import torch

from gpu_util import bf16_to_dev, bits_of, to_dev
from oracle import codecs, moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -8                 # half a bf16 step relative to the value
TINY = 2.0 ** -133            # one bf16 subnormal step


@pytest.mark.parametrize("t,topk,n", [(1, 1, 8), (7, 2, 33), (64, 8, 264), (700, 3, 2056)])
def test_gradient_of_the_combine(t, topk, n):
    import quantized_gemm_int4_amd as hm
    r = np.random.default_rng([t, topk, n])
    y, dout = (codecs.bf16_rne_bits(r.normal(0, 1, s).astype(np.float32)) for s in ((t * topk, n), (t, n)))
    w = r.random((t, topk)).astype(np.float32)
    own = torch.arange(t * topk, dtype=torch.int32, device="cuda").reshape(t, topk)
    yd, wd = bf16_to_dev(y), to_dev(w)
    if n % 8 == 0:
        out = hm.hm_moe_combine(yd, wd, topk)
        assert torch.equal(hm.hm_moe_collect(yd, wd, own).view(torch.int16), out.view(torch.int16))
    dy, dw = hm.hm_moe_collect_grad(bf16_to_dev(dout), yd, wd, own)
    val = lambda b: codecs.bf16_value(b).astype(np.float64)                               # noqa: E731
    rdy, rdw, bdw = moe.collect_grad_ref(val(dout), val(y), w, own.cpu().numpy())
    # one fp32 rounding of the product and one to bf16; n products summed in fp32, 2^-24 an addition, taken twice
    assert (np.abs(val(bits_of(dy)) - rdy) <= U * np.abs(rdy) * (1 + 2.0 ** -8) + TINY).all()
    assert (np.abs(dw.cpu().numpy() - rdw) <= (n + 8) * 2.0 ** -23 * bdw).all()
