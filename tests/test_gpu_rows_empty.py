"""A dispatch of no tokens, as a rank of an expert-parallel job may have: its
counts and offsets say so."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("side", [False, True])
def test_dispatch_of_no_tokens_counts_none(given, side):
    import quantized_gemm_int4_amd as hm
    E, i32 = 5, torch.int32
    x, ids = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 2, dtype=i32, device="cuda")
    torch.full((1 << 12,), 7, dtype=i32, device="cuda")         # what a new array may find in its memory
    kw = dict(counts=torch.full((E,), 7, dtype=i32, device="cuda"),
              offsets=torch.full((E + 1,), 7, dtype=i32, device="cuda")) if given else {}
    stream = torch.cuda.Stream() if side else None
    if side:
        stream.wait_stream(torch.cuda.current_stream())
    xs, counts, offsets, pairs, pos = hm.hm_moe_dispatch(x, ids, E, stream=stream, **kw)
    if side:
        stream.synchronize()
    assert counts.tolist() == [0] * E and offsets.tolist() == [0] * (E + 1)
    assert xs.shape == (0, 64) and pairs.shape == (0,) and pos.shape == (0, 2)
    with pytest.raises(hm.HmError):
        hm.hm_moe_dispatch(x, ids, 1)                           # topk above the experts
