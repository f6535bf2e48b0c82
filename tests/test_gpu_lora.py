"""GPU parity of the low-rank adapters and their gradient against the oracle's
fp64 definition, element by element.

Error bounds, from the arithmetic (u = 2^-8 is half a bf16 step relative to
the value, S the oracle's sum of absolute terms): the result is rounded to
bf16 once (u |y|); h or g enters the second product as two bf16 terms, off by
at most 2^-16 of it (2^-16 S); the fp32 sums of K, N, rank or M terms are off
by at most 2^-24 S per addition, taken twice for the matrix unit's own
rounding."""
import numpy as np
import pytest
import torch

import synthetic
from gpu_util import bf16_to_dev, bits_of, quantize_experts, std_to_dev, to_dev
from oracle import codecs, lora, quant

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
TINY = 2.0 ** -120            # products of bf16 values that underflow in fp32, and bf16's own subnormal step

# m, n, k, rank, adapters
SHAPES = [(1, 1, 128, 8, 1), (1, 130, 256, 16, 3), (2, 16, 128, 128, 2), (5, 37, 256, 24, 3), (17, 64, 1152, 32, 17),
          (33, 130, 384, 40, 4), (64, 513, 128, 64, 2), (100, 256, 640, 96, 5), (130, 1023, 256, 128, 3),
          (300, 88, 256, 48, 512), (257, 640, 512, 16, 1), (4500, 40, 128, 8, 7),
          (16, 2500, 256, 64, 9), (150, 72, 256, 16, 6), (150, 300, 256, 32, 6), (150, 72, 128, 64, 6),
          (1500, 200, 256, 128, 3), (1100, 130, 128, 64, 2), (48, 2600, 128, 16, 30)]


def _bits(r, *shape, std=1.0):
    return codecs.bf16_rne_bits(r.normal(0, std, shape).astype(np.float32))


def _val(bits):
    return codecs.bf16_value(bits).astype(np.float64)


def _case(m, n, k, rank, L, seed=0, none=0.2):
    r = np.random.default_rng([m, n, k, rank, L, seed])
    c = dict(x=_bits(r, m, k), a=_bits(r, L, rank, k, std=k ** -0.5), b=_bits(r, L, n, rank, std=0.3),
             base=_bits(r, m, n), dy=_bits(r, m, n), dxb=_bits(r, m, k),
             s=r.normal(0, 1.5, L).astype(np.float32), ids=r.integers(0, L, m).astype(np.int32))
    if none and m > 1:
        c["ids"][r.random(m) < none] = -1
        c["ids"][0] = L
        c["ids"][m // 2] = np.iinfo(np.int32).min
        c["ids"][m - 1] = 0
    return c


def _dev(c):
    return {k: bf16_to_dev(v) if v.dtype == np.uint16 else to_dev(v) for k, v in c.items()}


def _check_fwd(c, y, h, k, rank, base=True):
    (ry, rh), (by, bh) = lora.lora_ref(_val(c["x"]), c["ids"], _val(c["a"]), _val(c["b"]), c["s"],
                                       _val(c["base"]) if base else None)
    e = by * (2.0 ** -16 + (k + 2 * rank + 64) * 2.0 ** -23)
    assert (np.abs(_val(bits_of(y)) - ry) <= U * (np.abs(ry) + e) + e + TINY).all()
    if h is not None:
        assert (np.abs(h.cpu().numpy() - rh) <= bh * (k + 64) * 2.0 ** -23 + TINY).all()


@pytest.mark.parametrize("m,n,k,rank,L", SHAPES)
def test_lora_parity(m, n, k, rank, L):
    import quantized_gemm_int4_amd as hm
    c = _case(m, n, k, rank, L)
    d, t = hm.lora_desc(n, k, rank, L), _dev(c)
    h = torch.full((m, rank), 9.0, device="cuda")
    y = hm.hm_lora(d, t["x"], t["ids"], t["a"], t["b"], t["s"], base=t["base"], h=h)
    _check_fwd(c, y, h, k, rank)
    none = (c["ids"] < 0) | (c["ids"] >= L)
    assert np.array_equal(bits_of(y)[none], c["base"][none]) and (h.cpu().numpy()[none] == 0).all()
    y2 = hm.hm_lora(d, t["x"], t["ids"], t["a"], t["b"], t["s"], base=t["base"])          # h not kept
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
    yb = t["base"].clone()
    hm.hm_lora(d, t["x"], t["ids"], t["a"], t["b"], t["s"], base=yb, y=yb)                # in place
    assert torch.equal(y.view(torch.int16), yb.view(torch.int16))
    y0 = hm.hm_lora(d, t["x"], t["ids"], t["a"], t["b"], t["s"])                          # no base
    _check_fwd(c, y0, None, k, rank, base=False)
    assert (bits_of(y0)[none] == 0).all()


def _check_grad(c, got, n, rank, dxb=True):
    h = c["h"]
    refs, bnds = lora.lora_grad_ref(_val(c["dy"]), _val(c["x"]), h, c["ids"], _val(c["a"]), _val(c["b"]), c["s"],
                                    _val(c["dxb"]) if dxb else None)
    m = len(c["ids"])
    terms = (n + 2 * rank + 64, n + m + 64, m + 64)
    for name, g, r, b, k in zip(("dx", "da", "db"), got, refs, bnds, terms):
        if g is None:
            continue
        e = b * (2.0 ** -16 + k * 2.0 ** -23)
        bad = np.abs(_val(bits_of(g)) - r) > U * (np.abs(r) + e) + e + TINY
        assert not bad.any(), (name, int(bad.sum()))


@pytest.mark.parametrize("m,n,k,rank,L", SHAPES)
def test_lora_grad_parity(m, n, k, rank, L):
    import quantized_gemm_int4_amd as hm
    c = _case(m, n, k, rank, L, seed=1)
    c["h"] = np.random.default_rng(m).normal(0, 1, (m, rank)).astype(np.float32)
    d, t = hm.lora_desc(n, k, rank, L), _dev(c)
    args = (d, t["dy"], t["x"], t["h"], t["ids"], t["a"], t["b"], t["s"])
    sent = lambda *s: torch.full(s, 9.0, dtype=torch.bfloat16, device="cuda")             # noqa: E731
    got = hm.hm_lora_grad(*args, dx_base=t["dxb"], dx=sent(m, k), da=sent(L, rank, k), db=sent(L, n, rank))
    _check_grad(c, got, n, rank)
    unused = np.setdiff1d(np.arange(L), c["ids"])
    assert (bits_of(got[1])[unused] == 0).all() and (bits_of(got[2])[unused] == 0).all()
    again = hm.hm_lora_grad(*args, dx_base=t["dxb"])
    for a, b in zip(got, again):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))                      # equal calls, equal bits
    dxb = t["dxb"].clone()
    inplace = hm.hm_lora_grad(*args, dx_base=dxb, dx=dxb)
    assert torch.equal(inplace[0].view(torch.int16), got[0].view(torch.int16))
    bare = hm.hm_lora_grad(*args)
    _check_grad(c, bare, n, rank, dxb=False)
    no_dx = hm.hm_lora_grad(*args, need_dx=False)
    assert no_dx[0] is None and torch.equal(no_dx[1].view(torch.int16), got[1].view(torch.int16))


@pytest.mark.parametrize("m,ids", [(40, [2]), (700, [0]), (700, [-1]), (33, [0, 2]), (700, [0, 1, 2]), (2100, [1])])
def test_lora_rows_of_one_adapter_leave_the_others_alone(m, ids):
    """Every value of adapter 1, its rows of x, base, dy and its scale is NaN
    or infinite: rows of other adapters and rows without one are as without
    adapter 1, in both directions."""
    import quantized_gemm_int4_amd as hm
    n, k, rank, L = 136, 256, 16, 3
    c = _case(m, n, k, rank, L, seed=7, none=0)
    c["ids"] = np.resize(np.array(ids + [1, -1], dtype=np.int32), m)
    bad = c["ids"] == 1
    c["h"] = np.random.default_rng(2).normal(0, 1, (m, rank)).astype(np.float32)
    clean = {k2: v.copy() for k2, v in c.items()}
    for key in ("x", "base", "dy", "dxb"):
        c[key][bad] = 0x7FC0
    c["x"][bad, ::2] = 0x7F80
    c["h"][bad] = np.nan
    c["a"][1], c["b"][1], c["s"][1] = 0x7FC0, 0xFF80, np.nan
    d = hm.lora_desc(n, k, rank, L)
    out = []
    for cc in (clean, c):
        t = _dev(cc)
        h = torch.empty(m, rank, device="cuda")
        y = hm.hm_lora(d, t["x"], t["ids"], t["a"], t["b"], t["s"], base=t["base"], h=h)
        g = hm.hm_lora_grad(d, t["dy"], t["x"], t["h"], t["ids"], t["a"], t["b"], t["s"], dx_base=t["dxb"])
        out.append((bits_of(y)[~bad], h.cpu().numpy()[~bad], bits_of(g[0])[~bad], bits_of(g[1])[[0, 2]],
                    bits_of(g[2])[[0, 2]]))
    for a, b in zip(*out):
        assert np.array_equal(a, b)


def test_lora_no_rows_and_refusals():
    import quantized_gemm_int4_amd as hm
    d = hm.lora_desc(24, 128, 8, 2)
    bf, dev = torch.bfloat16, "cuda"
    z = lambda *s: torch.zeros(*s, dtype=bf, device=dev)                                  # noqa: E731
    a, b, s = z(2, 8, 128), z(2, 24, 8), torch.ones(2, device=dev)
    ids0, h0 = torch.empty(0, dtype=torch.int32, device=dev), torch.empty(0, 8, device=dev)
    assert hm.hm_lora(d, z(0, 128), ids0, a, b, s).shape == (0, 24)
    da, db = torch.ones(2, 8, 128, dtype=bf, device=dev), torch.ones(2, 24, 8, dtype=bf, device=dev)
    hm.hm_lora_grad(d, z(0, 24), z(0, 128), h0, ids0, a, b, s, da=da, db=db)
    assert (da == 0).all() and (db == 0).all()
    x, ids, h = z(3, 128), torch.zeros(3, dtype=torch.int32, device=dev), torch.zeros(3, 8, device=dev)
    for bad in (lambda: hm.hm_lora(d, x.float(), ids, a, b, s), lambda: hm.hm_lora(d, x[:, :64], ids, a, b, s),
                lambda: hm.hm_lora(d, x, ids.long(), a, b, s), lambda: hm.hm_lora(d, x, ids[:2], a, b, s),
                lambda: hm.hm_lora(d, x, ids, a.transpose(0, 1), b, s), lambda: hm.hm_lora(d, x, ids, a, b, s.half()),
                lambda: hm.hm_lora(d, x, ids, a, b, s, base=z(3, 25)), lambda: hm.hm_lora(d, x, ids, a, b, s, h=h[:2]),
                lambda: hm.hm_lora_grad(d, z(3, 23), x, h, ids, a, b, s),
                lambda: hm.hm_lora_grad(d, z(3, 24), x, h, ids, a, b, s, need_dx=False, dx_base=x)):
        with pytest.raises(ValueError):
            bad()
    ids100, need = torch.zeros(100, dtype=torch.int32, device=dev), hm.hm_lora_workspace_size(d, 100)
    assert need > 0
    with pytest.raises(hm.HmError):
        hm.hm_lora(d, z(100, 128), ids100, a, b, s, ws=torch.empty(need - 1, dtype=torch.uint8, device=dev))
    with pytest.raises(hm.HmError):
        hm.hm_lora_workspace_size(hm.lora_desc(24, 128, 12, 2), 4)


@pytest.mark.parametrize("m", [3, 60, 900])
def test_lora_in_a_graph_and_one_workspace_for_many_calls(m):
    """Forward and gradient captured once, replayed on new rows and ids with
    eager calls on the same workspace between the replays."""
    import quantized_gemm_int4_amd as hm
    n, k, rank, L = 200, 384, 24, 6
    t = _dev(_case(m, n, k, rank, L, seed=3))
    d = hm.lora_desc(n, k, rank, L)
    ws = torch.empty(max(hm.hm_lora_workspace_size(d, m), hm.hm_lora_grad_workspace_size(d, m), 256), dtype=torch.uint8,
                     device="cuda")

    def step():
        h = torch.empty(m, rank, device="cuda")
        y = hm.hm_lora(d, t["x"], t["ids"], t["a"], t["b"], t["s"], base=t["base"], h=h, ws=ws)
        return (y,) + hm.hm_lora_grad(d, t["dy"], t["x"], h, t["ids"], t["a"], t["b"], t["s"], dx_base=t["dxb"], ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i in range(3):
        new = _dev(_case(m, n, k, rank, L, seed=10 + i, none=0.3 * i))
        for key in t:
            t[key].copy_(new[key])
        ws.fill_(0xA5)                                          # nothing in it outlives a call
        want = [v.clone() for v in step()]
        ws.fill_(0x5A)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("m", [2, 50, 400])
def test_lora_calls_on_two_streams_at_once(m):
    """Two streams run forward and gradient of different rows side by side,
    each with buffers of its own; the bits are those of the same calls alone."""
    import quantized_gemm_int4_amd as hm
    n, k, rank, L = 300, 512, 32, 4
    d = hm.lora_desc(n, k, rank, L)
    cases = [_dev(_case(m, n, k, rank, L, seed=20 + i)) for i in range(2)]

    def step(t, stream=None):
        h = torch.zeros(m, rank, device="cuda") if stream is None else t["hbuf"]
        y = hm.hm_lora(d, t["x"], t["ids"], t["a"], t["b"], t["s"], base=t["base"], h=h, stream=stream)
        return (y,) + hm.hm_lora_grad(d, t["dy"], t["x"], h, t["ids"], t["a"], t["b"], t["s"], stream=stream)

    want = [step(t) for t in cases]
    for t in cases:
        t["hbuf"] = torch.zeros(m, rank, device="cuda")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[step(t, s) for t, s in zip(cases, streams)] for _ in range(5)][-1]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for a, b in zip(w, g):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("m", [1, 20, 300])
def test_adapters_beside_the_low_bit_projection(m):
    """As a layer runs: the shared INT4 projection, the adapters added in
    place on its output, then the gradient of that step."""
    import quantized_gemm_int4_amd as hm
    n, k, rank, L = 272, 512, 16, 5
    codes, scales, zeros, _ = quantize_experts(quant.FMT_INT4_SYM, [synthetic.weights(3, n, k)])
    dw = hm.wdesc(quant.FMT_INT4_SYM, n, k)
    w = hm.hm_transform(dw, *std_to_dev(quant.FMT_INT4_SYM, codes, scales, zeros))
    c = _case(m, n, k, rank, L, seed=5)
    t, d = _dev(c), hm.lora_desc(n, k, rank, L)
    y = hm.hm_gemm(dw, w, t["x"])
    c["base"] = bits_of(y).copy()
    h = torch.empty(m, rank, device="cuda")
    hm.hm_lora(d, t["x"], t["ids"], t["a"], t["b"], t["s"], base=y, y=y, h=h)
    _check_fwd(c, y, h, k, rank)
    c["h"] = h.cpu().numpy()
    got = hm.hm_lora_grad(d, t["dy"], t["x"], h, t["ids"], t["a"], t["b"], t["s"], dx_base=t["dxb"])
    _check_grad(c, got, n, rank)


@pytest.mark.parametrize("m,n,k,rank,L", [(1, 14336, 4096, 16, 64), (48, 7168, 2048, 64, 64), (700, 4096, 7168, 32, 9),
                                              (64, 14336, 512, 16, 64), (300001, 24, 128, 8, 5), (20000, 256, 128, 32, 3)])
def test_lora_layer_shapes_sampled(m, n, k, rank, L):
    """Layer-sized calls against fp64 products on the GPU; the second half of
    the adapters is not used by any row."""
    import quantized_gemm_int4_amd as hm
    g = torch.Generator(device="cuda").manual_seed(m)
    rn = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)   # noqa: E731
    x, a, b, base, dy = rn(m, k), rn(L, rank, k, std=k ** -0.5), rn(L, n, rank, std=0.02), rn(m, n), rn(m, n)
    s = torch.rand(L, generator=g, device="cuda") + 0.5
    ids = torch.randint(0, (L + 1) // 2, (m,), generator=g, device="cuda", dtype=torch.int32)
    d = hm.lora_desc(n, k, rank, L)
    h = torch.empty(m, rank, device="cuda")
    y = hm.hm_lora(d, x, ids, a, b, s, base=base, h=h)
    dx, da, db = hm.hm_lora_grad(d, dy, x, h, ids, a, b, s)
    f = torch.float64
    for e in range(L):
        r = (ids == e).nonzero()[:, 0]
        if r.numel() == 0:
            assert (da[e] == 0).all() and (db[e] == 0).all()
            continue
        A, B, X, D, H = a[e].to(f), b[e].to(f), x[r].to(f), dy[r].to(f), h[r].to(f)
        hr = s[e].to(f) * (X @ A.t())
        G = s[e].to(f) * (D @ B)
        ab = lambda p, q: p.abs() @ q.abs()                                               # noqa: E731
        Hb, Gb = s[e].to(f) * ab(X, A.t()), s[e].to(f) * ab(D, B)
        for got, ref, bnd, terms in ((y[r], base[r].to(f) + hr @ B.t(), base[r].to(f).abs() + ab(Hb, B.t()), k + 2 * rank),
                                     (dx[r], G @ A, ab(Gb, A), n + 2 * rank), (da[e], G.t() @ X, ab(Gb.t(), X), n + m),
                                     (db[e], D.t() @ H, ab(D.t(), H), m)):
            err = bnd * (2.0 ** -16 + (terms + 64) * 2.0 ** -23)
            assert ((got.to(f) - ref).abs() <= U * (ref.abs() + err) + err).all()


def test_lora_rows_beyond_4gib():
    """base, y and dy past 2^32 bytes: the last rows of y, and db of some
    columns (a sum over every row), against fp64."""
    import quantized_gemm_int4_amd as hm
    m, n, k, rank, L = 160000, 14336, 128, 8, 2                 # 4.6 GB of y
    g = torch.Generator(device="cuda").manual_seed(4)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)     # noqa: E731
    x, a, b, y, s = rn(m, k), rn(L, rank, k), rn(L, n, rank), rn(m, n), torch.ones(L, device="cuda")
    ids = torch.arange(m, device="cuda", dtype=torch.int32) % 3 - 1                       # a third without an adapter
    d, h, f = hm.lora_desc(n, k, rank, L), torch.empty(m, rank, device="cuda"), torch.float64
    last = slice(m - 300, m)
    base = y[last].clone()
    hm.hm_lora(d, x, ids, a, b, s, base=y, y=y, h=h)
    e = ids[last].long().clamp(min=0)
    on = (ids[last] >= 0).to(f)[:, None]
    hr = on * torch.stack([a[i].to(f) @ v.to(f) for i, v in zip(e, x[last])])
    hb = on * torch.stack([a[i].to(f).abs() @ v.to(f).abs() for i, v in zip(e, x[last])])
    ref = base.to(f) + torch.stack([b[i].to(f) @ v for i, v in zip(e, hr)])
    bnd = base.to(f).abs() + torch.stack([b[i].to(f).abs() @ v for i, v in zip(e, hb)])
    err = bnd * (2.0 ** -16 + (k + 2 * rank + 64) * 2.0 ** -23)
    assert ((y[last].to(f) - ref).abs() <= U * (ref.abs() + err) + err).all()
    _, _, db = hm.hm_lora_grad(d, y, x, h, ids, a, b, s, need_dx=False)
    cols = torch.tensor([0, 1, 129, n - 1], device="cuda")
    for i in range(L):
        r = (ids == i).nonzero()[:, 0]
        dy = y[r][:, cols].to(f)
        ref, bnd = dy.t() @ h[r].to(f), dy.t().abs() @ h[r].to(f).abs()
        # the terms of one sum are added in four waves' and sixteen chunks' pieces of 32 rows a step
        err = bnd * (2.0 ** -16 + (m + 64) * 2.0 ** -23)
        assert ((db[i][cols].to(f) - ref).abs() <= U * (ref.abs() + err) + err).all()
