"""Batches without rows in the gradient of the 8-bit integer layers."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _layer(n, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    x8, sx = torch.zeros(0, k, dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda")
    w8 = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    return torch.zeros(0, n, dtype=torch.bfloat16, device="cuda"), x8, sx, w8, torch.rand(n, generator=g, device="cuda")


@pytest.mark.parametrize("n", [64, 257])
def test_dx_alone(n):
    """Frozen weights: an empty dx, given or not."""
    import quantized_gemm_int4_amd as hm
    a = _layer(n, 256)
    dx, dw = hm.hm_gemm_int8_grad(*a, need_dw=False)
    assert dx.shape == (0, 256) and dw is None
    own = torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda")
    assert hm.hm_gemm_int8_grad(*a, dx=own, need_dw=False)[0] is own
    with pytest.raises(ValueError):                            # its shape is checked all the same
        hm.hm_gemm_int8_grad(*a, dx=torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda"), need_dw=False)
    with pytest.raises(hm.HmError):                            # neither gradient is wanted
        hm.hm_gemm_int8_grad(*a, need_dx=False, need_dw=False)
    with pytest.raises(hm.HmError):                            # nor are its sizes taken on trust
        hm.hm_gemm_int8_grad(*_layer(n, 200), need_dw=False)
