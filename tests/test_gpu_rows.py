"""GPU parity of the rows in expert order: the dispatch is exact, the collect
and both gradients match the oracle's fp64 sums element by element, and a
block run through them gives the bits of the pair-order path.

Error bounds (u = 2^-8, half a bf16 step relative to the value): one rounding
of the result plus the fp32 sum of topk (or n) products, each addition off by
at most 2^-24 of the sum of absolute terms, taken twice."""
import numpy as np
import pytest
import torch

import synthetic
from gpu_util import bf16_to_dev, bits_of, quantize_experts, std_to_dev, to_dev
from oracle import codecs, moe, quant

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
TINY = 2.0 ** -133            # one bf16 subnormal step


def _rows(r, m, n):
    return codecs.bf16_rne_bits(r.normal(0, 2, (m, n)).astype(np.float32))


def _val(bits):
    return codecs.bf16_value(bits).astype(np.float64)


# one token, one wave, many tokens, chunked sorts; rows shorter than a chunk, odd, a chunk past a block's first pass
SHAPES = [(1, 1, 1, 1), (1, 8, 16, 7168), (3, 2, 5, 7), (5, 3, 9, 13), (64, 8, 256, 264), (33, 6, 512, 2049),
          (70, 9, 40, 2056), (300, 17, 60, 72), (600, 8, 256, 40), (5000, 1, 3, 24), (2500, 4, 64, 33), (2, 512, 512, 130),
          (1024, 1, 7, 40), (1025, 1, 7, 40), (128, 8, 512, 16), (33000, 4, 100, 8)]


def _ids(r, t, topk, E, dropped):
    ids = r.integers(0, E, (t, topk)).astype(np.int32)
    if dropped:
        ids[r.random((t, topk)) < dropped] = -1
        flat = ids.reshape(-1)
        flat[:2] = [E, np.iinfo(np.int32).min][:flat[:2].size]
    return ids


@pytest.mark.parametrize("dropped", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("t,topk,E,n", SHAPES)
def test_dispatch_exact(t, topk, E, n, dropped):
    import quantized_gemm_int4_amd as hm
    r = np.random.default_rng([t, topk, E, n, int(10 * dropped)])
    ids = _ids(r, t, topk, E, dropped)
    if dropped == 1.0:
        ids[:] = -1
    x = _rows(r, t, n)
    x.reshape(-1)[0] = 0x7FC0                                   # a NaN and an infinity are only moved
    x.reshape(-1)[-1] = 0xFF80
    P = t * topk
    xs = torch.full((P, n), 7.0, dtype=torch.bfloat16, device="cuda")
    sp = torch.full((P,), -5, dtype=torch.int32, device="cuda")
    got = hm.hm_moe_dispatch(bf16_to_dev(x), to_dev(ids), E, xs=xs, sorted_pairs=sp)
    pos, off = moe.positions_ref(ids, E)
    live = int(off[-1])
    inv = np.full(P, -5, dtype=np.int32)
    inv[pos.ravel()[pos.ravel() >= 0]] = np.nonzero(pos.ravel() >= 0)[0]
    assert np.array_equal(got[4].cpu().numpy(), pos)
    assert np.array_equal(got[2].cpu().numpy(), off)
    assert np.array_equal(got[1].cpu().numpy(), np.diff(off))
    assert np.array_equal(got[3].cpu().numpy(), inv)            # entries behind the last pair left as they were
    want = np.full((P, n), 0x40E0, dtype=np.uint16)
    want[:live] = x[inv[:live] // topk]
    assert np.array_equal(bits_of(got[0]), want)


@pytest.mark.parametrize("dropped", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("t,topk,E,n", SHAPES)
def test_collect_and_gradients(t, topk, E, n, dropped):
    import quantized_gemm_int4_amd as hm
    r = np.random.default_rng([n, t, topk, E, int(10 * dropped)])
    ids = _ids(r, t, topk, E, dropped)
    if dropped == 1.0:
        ids[:] = -1
    pos, off = moe.positions_ref(ids, E)
    P, live = t * topk, int(off[-1])
    ys, dout = _rows(r, P, n), _rows(r, t, n)
    ys[live:] = 0x7FC0                                          # rows that no pair names hold NaN
    w = r.normal(0, 1, (t, topk)).astype(np.float32)
    w[pos < 0] = np.nan                                         # weights of dropped pairs are not used
    posd, yd, wd, dd = to_dev(pos), bf16_to_dev(ys), to_dev(w), bf16_to_dev(dout)

    out = hm.hm_moe_collect(yd, wd, posd)
    ref, bnd = moe.collect_ref(_val(ys), w, pos)
    e = np.abs(_val(bits_of(out)) - ref)
    sum_err = topk * 2.0 ** -23 * bnd
    assert (e <= U * (np.abs(ref) + sum_err) + sum_err + TINY).all()

    dx = hm.hm_moe_dispatch_grad(yd, posd)
    ref, bnd = moe.collect_ref(_val(ys), None, pos)
    e = np.abs(_val(bits_of(dx)) - ref)
    sum_err = topk * 2.0 ** -23 * bnd
    assert (e <= U * (np.abs(ref) + sum_err) + sum_err + TINY).all()

    rdys, rdw, bdw = moe.collect_grad_ref(_val(dout), _val(ys), w, pos)
    for inplace in (False, True):
        dst = yd.clone() if inplace else torch.full((P, n), 7.0, dtype=torch.bfloat16, device="cuda")
        before = bits_of(dst)
        dys, dw = hm.hm_moe_collect_grad(dd, dst if inplace else yd, wd, posd, dys=dst)
        gb = bits_of(dys)
        assert np.array_equal(gb[live:], before[live:])         # rows behind the last pair left as they were
        e = np.abs(_val(gb[:live]) - rdys[:live])
        # the product is one fp32 rounding, the result one bf16 rounding of it
        assert (e <= U * np.abs(rdys[:live]) * (1 + 2.0 ** -8) + TINY).all()
        assert (np.abs(dw.cpu().numpy() - rdw) <= (n + 8) * 2.0 ** -23 * bdw).all()
        assert (dw.cpu().numpy()[pos < 0] == 0).all()


def test_collect_ignores_positions_out_of_range_and_takes_equal_ones():
    import quantized_gemm_int4_amd as hm
    ys = bf16_to_dev(_rows(np.random.default_rng(1), 6, 40))
    pos = to_dev(np.array([[2, 2], [6, -7], [0, 2 ** 31 - 1]], dtype=np.int32))
    w = to_dev(np.array([[0.25, 0.5], [1, 1], [2, 1]], dtype=np.float32))
    out = hm.hm_moe_collect(ys, w, pos).float()
    want = torch.stack([ys[2].float() * 0.75, torch.zeros(40, device="cuda"), ys[0].float() * 2])
    assert (out - want).abs().max() <= U * want.abs().max()
    assert (out[1] == 0).all()
    dys, dw = hm.hm_moe_collect_grad(torch.ones(3, 40, dtype=torch.bfloat16, device="cuda"), ys, w,
                                     to_dev(np.array([[2, 3], [6, -7], [0, 2 ** 31 - 1]], dtype=np.int32)))
    assert (dys[[1, 4, 5]] == 0).all() and (dys[3] == 0.5).all() and dw[1].tolist() == [0.0, 0.0]


def test_rows_no_tokens_and_refusals():
    import quantized_gemm_int4_amd as hm
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    assert hm.hm_moe_dispatch(x, ids, 4)[0].shape == (0, 64)
    assert hm.hm_moe_collect(x, torch.empty(0, 2, device="cuda"), ids).shape == (0, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.ones(4, 2, device="cuda")
    ys = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: hm.hm_moe_dispatch(x.float(), ids, 4), lambda: hm.hm_moe_dispatch(x[:, ::2], ids, 4),
                lambda: hm.hm_moe_dispatch(x, ids.long(), 4), lambda: hm.hm_moe_dispatch(x, ids[:3], 4),
                lambda: hm.hm_moe_dispatch(x, ids, 4, xs=ys[:7]), lambda: hm.hm_moe_collect(ys[:7], w, ids),
                lambda: hm.hm_moe_collect(ys, w.double(), ids), lambda: hm.hm_moe_collect_grad(x[:3], ys, w, ids),
                lambda: hm.hm_moe_collect_grad(x, ys, w, ids, dys=x), lambda: hm.hm_moe_dispatch_grad(x, ids),
                lambda: hm.hm_moe_dispatch(x, ids.flatten(), 4), lambda: hm.hm_moe_dispatch_grad(ys, ids.flatten())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(hm.HmError):
        hm.hm_moe_dispatch(x, ids, 1)                           # topk above the experts


@pytest.mark.parametrize("t", [40, 2100])
def test_rows_on_another_stream_and_in_a_graph(t):
    """The whole round trip captured once and replayed with new inputs, eager
    calls between the replays; equal bits each time."""
    import quantized_gemm_int4_amd as hm
    topk, E, n = 4, 16, 520
    r = np.random.default_rng(t)
    x, ids = bf16_to_dev(_rows(r, t, n)), to_dev(_ids(r, t, topk, E, 0.2))
    w, dout = to_dev(r.random((t, topk)).astype(np.float32)), bf16_to_dev(_rows(r, t, n))

    def chain():
        xs, c, o, sp, pos = hm.hm_moe_dispatch(x, ids, E)
        out = hm.hm_moe_collect(xs, w, pos)
        dys, dw = hm.hm_moe_collect_grad(dout, xs, w, pos)
        return out, dw, hm.hm_moe_dispatch_grad(dys, pos), pos, c

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain()
    for i in range(3):
        x.copy_(bf16_to_dev(_rows(r, t, n)))
        ids.copy_(to_dev(_ids(r, t, topk, E, 0.3 * i)))
        want = chain()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else a.dtype),
                               b.view(torch.int16 if b.dtype == torch.bfloat16 else b.dtype))
    with_stream = hm.hm_moe_dispatch(x, ids, E, stream=side)
    side.synchronize()
    assert torch.equal(with_stream[4], want[3])


@pytest.mark.parametrize("fmt", [quant.FMT_INT4_SYM, quant.FMT_MXFP4])
def test_moe_block_in_expert_order_equals_pair_order(fmt):
    """dispatch, grouped GEMM on the expert-ordered rows (identity pairs),
    collect: the bits of sort, grouped GEMM in pair order, combine; and the
    backward pass of both ends against the oracle on the GPU's own values."""
    import quantized_gemm_int4_amd as hm
    t, topk, E, K, N = 50, 2, 6, 256, 160
    ids, w = synthetic.router_topk(6, t, E, topk)
    codes, scales, zeros, _ = quantize_experts(fmt, [synthetic.weights(16, N, K, index=e) for e in range(E)])
    d = hm.wdesc(fmt, N, K, E)
    wd = hm.hm_transform(d, *std_to_dev(fmt, codes, scales, zeros))
    x, idsd, wdev = bf16_to_dev(synthetic.activations(16, t, K, index=1)), to_dev(ids), to_dev(w)
    _, off, sp = hm.hm_moe_sort(idsd, E)
    want = hm.hm_moe_combine(hm.hm_moe_gemm(d, wd, x, off, sp, t, topk, 0), wdev, topk)
    xs, _, off2, sp2, pos = hm.hm_moe_dispatch(x, idsd, E)
    assert torch.equal(off, off2) and torch.equal(sp, sp2)
    same = torch.arange(t * topk, dtype=torch.int32, device="cuda")
    ys = hm.hm_moe_gemm(d, wd, xs, off2, same, t * topk, 1, 1)
    out = hm.hm_moe_collect(ys, wdev, pos)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    dout = bf16_to_dev(_rows(np.random.default_rng(3), t, N))
    dys, dw = hm.hm_moe_collect_grad(dout, ys, wdev, pos)
    _, rdw, bdw = moe.collect_grad_ref(_val(bits_of(dout)), _val(bits_of(ys)), w, pos.cpu().numpy())
    assert (np.abs(dw.cpu().numpy() - rdw) <= (N + 8) * 2.0 ** -23 * bdw).all()
    dxs = dys[:, :K // 2].contiguous()                          # any expert-ordered gradient
    dx = hm.hm_moe_dispatch_grad(dxs, pos)
    ref, bnd = moe.collect_ref(_val(bits_of(dxs)), None, pos.cpu().numpy())
    assert (np.abs(_val(bits_of(dx)) - ref) <= U * (np.abs(ref) + bnd * 2.0 ** -22) + bnd * 2.0 ** -22 + TINY).all()


def test_dispatch_rows_beyond_4gib():
    """Rows past 2^32 bytes of the expert-ordered array, sampled."""
    import quantized_gemm_int4_amd as hm
    t, topk, E, n = 40000, 8, 64, 7168                          # 4.6 GB of rows
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(t, n, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, E, (t, topk), generator=g, device="cuda", dtype=torch.int32)
    xs, _, off, sp, pos = hm.hm_moe_dispatch(x, ids, E)
    assert int(off[-1]) == t * topk
    assert torch.equal(torch.sort(pos.flatten()).values, torch.arange(t * topk, device="cuda", dtype=torch.int32))
    for lo in (0, t * topk // 2, t * topk - 3000):
        assert torch.equal(xs[lo:lo + 3000], x[(sp[lo:lo + 3000] // topk).long()])
    w = torch.zeros(t, topk, device="cuda")
    w[:, 3] = 1.0
    out = hm.hm_moe_collect(xs, w, pos)
    assert torch.equal(out, x)                                  # each token's own row back, bit for bit
