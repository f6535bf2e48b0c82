"""GPU parity of the 8-bit integer layers, their gated block and gradients with
the fp64 oracle, element by element.

Error bounds.  u = 2^-8 is half a bf16 step relative to the value, e = 2^-24
half an fp32 step.
  product: the integer sum is exact; its conversion and two products 3 e, the
    rounding u.
  gated: g and u off by 3 e each; silu's relative condition is at most 1 + |g|;
    its fast exponential and reciprocal (48 + |g|) 2 e; together (60 + 4 |g|) 2 e.
  gated gradient: the same for s and 1 - s; the terms 1 and g (1 - s) are added, so
    the bound of dg is in |dh u| s (1 + |g| (1 - s)).
  gradient: codes times scales are rounded to bf16 once (u of every term), n (m) fp32
    additions e of the sum of absolute terms each, the final rounding u."""
import numpy as np
import pytest
import torch

from gpu_util import bf16_to_dev, bits_of, to_dev
from oracle import codecs, int8

pytestmark = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24
TINY = 2.0 ** -126            # results this small may lose all bits on the way


def _val(bits):
    return codecs.bf16_value(bits).astype(np.float64)


def _bits(r, *shape, std=1.0):
    return codecs.bf16_rne_bits(r.normal(0, std, shape).astype(np.float32))


def _layer(r, m, n, k):
    """Codes of the whole int8 range with most weight near 0, scales over a factor of 1000."""
    q = lambda a, b: np.clip(np.rint(r.normal(0, 40, (a, b))), -128, 127).astype(np.int8)      # noqa: E731
    qx, qw = q(m, k), q(n, k)
    if m and n:
        qx[0, :3], qw[-1, -3:] = -128, -128
    sx = (10.0 ** r.uniform(-3, 0, m) / 40).astype(np.float32)
    sw = (10.0 ** r.uniform(-1.5, 0.5, n) / (40 * np.sqrt(k))).astype(np.float32)
    return qx, sx, qw, sw


def _dev(a):
    return [to_dev(v) for v in a]


def _close(got, ref, lim, what):
    y = _val(bits_of(got))
    bad = ~(np.abs(y - ref) <= lim)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), y[bad][:3], ref[bad][:3], lim[bad][:3])


ROWS = [1, 2, 5, 16, 17, 33, 64, 65, 127, 129, 300]


# ------------------------------------------------------------------ rows

@pytest.mark.parametrize("m,k", [(1, 1), (3, 7), (1, 128), (5, 129), (2, 512), (7, 520), (65, 1024), (4, 2056), (3, 4099),
                                 (2, 8192), (300, 384), (2, 14336), (3, 40000)])
def test_quant_rows(m, k):
    import quantized_gemm_int4_amd as hm
    r = np.random.default_rng([m, k])
    b = _bits(r, m, k)
    for i in range(min(m, 3)):                                 # exact halves of the largest value and odd halves of steps
        v = np.array([254.0, 127.0, 1.0, 3.0, -5.0, 253.0, -0.0])[:k].astype(np.float32) * np.float32(2.0 ** (i - 1))
        b[i, k - v.size:] = codecs.bf16_rne_bits(v)
    x8 = torch.full((m, k), 99, dtype=torch.int8, device="cuda")
    got, s = hm.hm_quant_int8_rows(bf16_to_dev(b), x8=x8)
    q, sr = int8.quant_rows(_val(b))
    assert np.array_equal(s.cpu().numpy(), sr)
    assert np.array_equal(got.cpu().numpy(), q)


def test_quant_every_pair_of_significands():
    """A row per largest significand and distance of exponents, a column per
    significand and sign: every ratio of two bf16 values down to code 0."""
    import quantized_gemm_int4_amd as hm
    sig = np.arange(128, 256)
    rows = []
    for shift in range(9):
        for a in sig:
            x = np.concatenate([sig, -sig]) * 2.0 ** -shift
            rows.append(np.concatenate([[float(a)], np.clip(x, -a, a) if shift == 0 else x]))
    x = np.array(rows, dtype=np.float32)
    for scale in (1.0, 2.0 ** -110, 2.0 ** 118):
        b = codecs.bf16_rne_bits(x * np.float32(scale))
        q, s = int8.quant_rows(_val(b))
        got, sg = hm.hm_quant_int8_rows(bf16_to_dev(b))
        assert np.array_equal(sg.cpu().numpy(), s), scale
        assert np.array_equal(got.cpu().numpy(), q), scale


def test_quant_far_magnitudes_and_rows_that_are_not_finite():
    import quantized_gemm_int4_amd as hm
    for k in (40, 264, 515):
        b = np.zeros((9, k), dtype=np.uint16)
        r = np.random.default_rng(k)
        b[0] = r.integers(0, 0x80, k)                          # subnormals
        b[1] = r.integers(0x7F00, 0x7F80, k)                   # up to the largest finite value
        b[2, 5], b[2, 7] = 1, 0x8001                           # the smallest of all
        b[3] = _bits(r, k)
        b[3, 3] = 0x7F80                                       # an infinity, NaN of either sign
        b[4, k - 1], b[5, 0], b[6, 1] = 0xFF80, 0x7FC0, 0xFF81
        b[8] = _bits(r, k, std=1e30)
        q, s = int8.quant_rows(_val(b))
        got, sg = hm.hm_quant_int8_rows(bf16_to_dev(b))
        assert np.array_equal(sg.cpu().numpy(), s, equal_nan=True)
        assert np.array_equal(got.cpu().numpy(), q)


# --------------------------------------------------------------- products

@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,k", [(1, 128), (16, 256), (100, 384), (129, 128), (257, 640), (512, 1152), (1030, 896)])
def test_product(m, n, k):
    import quantized_gemm_int4_amd as hm
    r = np.random.default_rng([m, n, k])
    a = _layer(r, m, n, k)
    ref = int8.product(*a)
    y = torch.full((m + 1, n), 7.0, dtype=torch.bfloat16, device="cuda")
    hm.hm_gemm_int8(*_dev(a), y=y[:m])
    _close(y[:m], ref, np.abs(ref) * (U + 4 * E) + TINY, "y")
    assert (y[m] == 7).all()                                   # rows behind the last are left alone


@pytest.mark.parametrize("m,n,k", [(1, 4096, 14336), (700, 900, 512), (1021, 515, 384), (513, 2049, 256), (2000, 1100, 128)])
def test_product_more_tiles(m, n, k):
    import quantized_gemm_int4_amd as hm
    a = _layer(np.random.default_rng([m, n, k]), m, n, k)
    ref = int8.product(*a)
    _close(hm.hm_gemm_int8(*_dev(a)), ref, np.abs(ref) * (U + 4 * E) + TINY, "y")


@pytest.mark.parametrize("m", [1, 40, 200, 1030])
def test_product_largest_sum(m):
    """k at its limit with every code at -128: the sum is 2^14 (2^17 - 2^7), just inside an int32."""
    import quantized_gemm_int4_amd as hm
    k, n = 130944, 33
    qx, qw = np.full((m, k), -128, np.int8), np.full((n, k), -128, np.int8)
    qx[:, 0] = 127
    s = np.full(max(m, n), 2.0 ** -20, np.float32)
    y = hm.hm_gemm_int8(to_dev(qx), to_dev(s[:m]), to_dev(qw), to_dev(s[:n]))
    ref = (128.0 * 128 * (k - 1) - 128 * 127) * 2.0 ** -40
    _close(y, np.full((m, n), ref), np.full((m, n), ref * (U + 4 * E)), "y")


@pytest.mark.parametrize("m", [3, 50, 150, 1030])
def test_scales_that_are_not_finite_stay_in_their_row_and_column(m):
    import quantized_gemm_int4_amd as hm
    n, k = 200, 256
    a = _layer(np.random.default_rng(m), m, n, k)
    a[1][1], a[3][7], a[3][199] = np.nan, np.inf, np.nan
    ref = int8.product(*a)
    y = _val(bits_of(hm.hm_gemm_int8(*_dev(a))))
    ok = np.ones((m, n), bool)
    ok[1], ok[:, 7], ok[:, 199] = False, False, False
    assert np.isnan(y[1]).all() and np.isnan(y[:, 199]).all() and not np.isfinite(y[:, 7]).any()
    assert (np.abs(y - ref)[ok] <= (np.abs(ref) * (U + 4 * E) + TINY)[ok]).all()


def _gated_lim(h, g):
    return np.abs(h) * (U + (60 + 4 * np.abs(g)) * 2 * E) + TINY


GATED = [(1, 128), (32, 256), (33, 128), (100, 384), (257, 640), (515, 896)]


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("d,k", GATED)
def test_gated(m, d, k):
    import quantized_gemm_int4_amd as hm
    r = np.random.default_rng([m, d, k, 1])
    a = _layer(r, m, 2 * d, k)
    a = (a[0], a[1] * 8, a[2], a[3])                           # gates up to about 60
    h, g, _ = int8.gated(*a)
    out = torch.full((m + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    hm.hm_gemm_int8_gated(*_dev(a), h=out[:m])
    _close(out[:m], h, _gated_lim(h, g), "h")
    assert (out[m] == 7).all()


@pytest.mark.parametrize("m", ROWS + [513])
@pytest.mark.parametrize("d,k", GATED)
def test_gated_gradient(m, d, k):
    import quantized_gemm_int4_amd as hm
    r = np.random.default_rng([m, d, k, 2])
    a = _layer(r, m, 2 * d, k)
    a = (a[0], a[1] * 8, a[2], a[3])
    dhb = _bits(r, m, d)
    dg, du, g, u = int8.gated_grad(_val(dhb), *a)
    out = torch.full((m + 1, 2 * d), 7.0, dtype=torch.bfloat16, device="cuda")
    hm.hm_gemm_int8_gated_grad(bf16_to_dev(dhb), *_dev(a), dgu=out[:m])
    c = (60 + 4 * np.abs(g)) * 2 * E
    big = np.abs(_val(dhb) * u) * int8.sigmoid(g) * (1 + np.abs(g) * int8.sigmoid(-g))
    _close(out[:m, d:].contiguous(), du, np.abs(du) * (U + c) + TINY, "du")
    _close(out[:m, :d].contiguous(), dg, np.abs(dg) * U + big * 2 * c + TINY, "dg")
    assert (out[m] == 7).all()


@pytest.mark.parametrize("m", [1, 20, 140, 1030])
def test_gates_far_out(m):
    """Gates to +-1e4 and beyond the exponential's range; a gate of exactly 0."""
    import quantized_gemm_int4_amd as hm
    d, k = 64, 128
    r = np.random.default_rng(m)
    qx = np.zeros((m, k), np.int8)
    qx[:, 0] = 1
    qw = np.zeros((2 * d, k), np.int8)
    qw[:d, 0] = np.linspace(-127, 127, d).astype(np.int8)
    qw[d:, 0] = r.integers(-127, 128, d)
    sw = np.where(np.arange(2 * d) < d, 100.0, 0.01).astype(np.float32)
    sx = np.ones(m, np.float32)
    a = (qx, sx, qw, sw)
    h, g, u = int8.gated(*a)
    _close(hm.hm_gemm_int8_gated(*_dev(a)), h, _gated_lim(h, g), "h")
    dhb = _bits(r, m, d)
    dg, du, _, _ = int8.gated_grad(_val(dhb), *a)
    out = hm.hm_gemm_int8_gated_grad(bf16_to_dev(dhb), *_dev(a))
    c = (60 + 4 * np.abs(g)) * 2 * E
    big = np.abs(_val(dhb) * u) * int8.sigmoid(g) * (1 + np.abs(g) * int8.sigmoid(-g))
    _close(out[:, d:].contiguous(), du, np.abs(du) * (U + c) + TINY, "du")
    _close(out[:, :d].contiguous(), dg, np.abs(dg) * U + big * 2 * c + TINY, "dg")


# --------------------------------------------------------------- gradients

def _check_grad(got, dyb, a, what):
    (dx, dw), (bx, bw) = int8.grad(_val(dyb), *a)
    m, n = dyb.shape
    for name, y, ref, b, terms in (("dx", got[0], dx, bx, n), ("dw", got[1], dw, bw, m)):
        if y is not None:
            _close(y, ref, b * (U + (terms + 2) * 2 * E) * (1 + U) + np.abs(ref) * U + TINY, (what, name))
            # under the worst case: the roundings of 16 terms and more are independent, at most u each, so their sum's
            # and the result's own have 2-norms of at most u / sqrt(3), 0.82 u together.  With one term a result nothing
            # averages out (equal codes are rounded alike, in every result) and only the worst case holds: the
            # term's rounding and the result's, (1 + u)^2 - 1 <= 2 u (1 + u).
            err, size = np.linalg.norm(_val(bits_of(y)) - ref), np.linalg.norm(ref)
            if terms == 1 or terms >= 16:
                assert err <= (U if terms >= 16 else 2 * U * (1 + U)) * size, (what, name, err / size)


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,k", [(1, 128), (16, 256), (72, 128), (100, 384), (129, 128), (256, 640), (515, 896)])
def test_gradient(m, n, k):
    import quantized_gemm_int4_amd as hm
    r = np.random.default_rng([m, n, k, 3])
    a, dyb = _layer(r, m, n, k), _bits(r, m, n, std=0.05)
    dx = torch.full((m + 1, k), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((n + 1, k), 7.0, dtype=torch.bfloat16, device="cuda")
    hm.hm_gemm_int8_grad(bf16_to_dev(dyb), *_dev(a), dx=dx[:m], dw=dw[:n])
    assert (dx[m] == 7).all() and (dw[n] == 7).all()
    _check_grad((dx[:m], dw[:n]), dyb, a, (m, n, k))


@pytest.mark.parametrize("m,n,k", [(700, 1500, 512), (1021, 515, 1152), (2300, 264, 128), (257, 4099, 256)])
def test_gradient_more_tiles(m, n, k):
    import quantized_gemm_int4_amd as hm
    r = np.random.default_rng([m, n, k, 4])
    a, dyb = _layer(r, m, n, k), _bits(r, m, n, std=0.05)
    _check_grad(hm.hm_gemm_int8_grad(bf16_to_dev(dyb), *_dev(a)), dyb, a, (m, n, k))


@pytest.mark.parametrize("m,n", [(20, 72), (300, 129)])
def test_gradient_of_one_side(m, n):
    import quantized_gemm_int4_amd as hm
    k = 256
    r = np.random.default_rng([m, n, k, 5])
    a, dyb = _layer(r, m, n, k), _bits(r, m, n)
    d, dy = _dev(a), bf16_to_dev(dyb)
    both = hm.hm_gemm_int8_grad(dy, *d)
    dx, none = hm.hm_gemm_int8_grad(dy, *d, need_dw=False)
    assert none is None and torch.equal(dx, both[0])
    none, dw = hm.hm_gemm_int8_grad(dy, *d, need_dx=False)
    assert none is None and torch.equal(dw, both[1])


@pytest.mark.parametrize("m,n", [(30, 72), (257, 100), (64, 129)])
def test_gradient_rows_and_columns_that_are_not_finite_stay_alone(m, n):
    """An infinity in dy: its row of dx and its row (channel) of dw; no other
    row or channel sees it, at sizes whose tiles are not full."""
    import quantized_gemm_int4_amd as hm
    k = 256
    r = np.random.default_rng([m, n, 6])
    a, dyb = _layer(r, m, n, k), _bits(r, m, n)
    dyb[1, n - 1] = 0x7F80
    dx, dw = (_val(bits_of(t)) for t in hm.hm_gemm_int8_grad(bf16_to_dev(dyb), *_dev(a)))
    assert np.isfinite(np.delete(dx, 1, 0)).all() and np.isfinite(dw[:n - 1]).all()
    assert not np.isfinite(dx[1]).all() and not np.isfinite(dw[n - 1]).all()


# ------------------------------------------------------------- empty calls

def test_no_rows():
    import quantized_gemm_int4_amd as hm
    x8, s = torch.zeros(0, 256, dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda")
    r = np.random.default_rng(0)
    _, _, qw, sw = _layer(r, 1, 66, 256)
    w8, sw = to_dev(qw), to_dev(sw)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q, qs = hm.hm_quant_int8_rows(torch.zeros(0, 256, **bf))
    assert q.shape == (0, 256) and qs.shape == (0,)
    assert hm.hm_gemm_int8(x8, s, w8, sw).shape == (0, 66)
    assert hm.hm_gemm_int8_gated(x8, s, w8, sw).shape == (0, 33)
    assert hm.hm_gemm_int8_gated_grad(torch.zeros(0, 33, **bf), x8, s, w8, sw).shape == (0, 66)
    dw = torch.full((66, 256), 7.0, **bf)
    dx, dw = hm.hm_gemm_int8_grad(torch.zeros(0, 66, **bf), x8, s, w8, sw, dw=dw)
    assert dx.shape == (0, 256) and not dw.any()


# ----------------------------------------------------- together, as in use

def _block(hm, x, wgu, wdn, dy):
    """One training step of a gated feed-forward block: bf16 rows and master
    weights in, output and gradients out; between the passes only 8-bit rows
    and scales are kept."""
    w8, sw = hm.hm_quant_int8_rows(wgu)
    v8, sv = hm.hm_quant_int8_rows(wdn)
    x8, sx = hm.hm_quant_int8_rows(x)
    h8, sh = hm.hm_quant_int8_rows(hm.hm_gemm_int8_gated(x8, sx, w8, sw))
    y = hm.hm_gemm_int8(h8, sh, v8, sv)
    dh, dwdn = hm.hm_gemm_int8_grad(dy, h8, sh, v8, sv)
    dgu = hm.hm_gemm_int8_gated_grad(dh, x8, sx, w8, sw)
    dx, dwgu = hm.hm_gemm_int8_grad(dgu, x8, sx, w8, sw)
    return y, dx, dwgu, dwdn


def _block_inputs(m, d, k, seed):
    r = np.random.default_rng(seed)
    return [bf16_to_dev(_bits(r, *s, std=std)) for s, std in (((m, k), 1.0), ((2 * d, k), k ** -0.5), ((k, d), d ** -0.5), ((m, k), 0.1))]


@pytest.mark.parametrize("m,d,k", [(1, 128, 256), (33, 256, 384), (300, 640, 256)])
def test_block_step(m, d, k):
    """Every stage against the oracle on the stage's own inputs, and the whole
    against the block in fp64 without any quantization: codes are off by at most
    half a step of amax / 127, so rows differ by a few per cent."""
    import quantized_gemm_int4_amd as hm
    x, wgu, wdn, dy = _block_inputs(m, d, k, [m, d, k])
    y, dx, dwgu, dwdn = _block(hm, x, wgu, wdn, dy)
    f = lambda t: t.cpu().double().requires_grad_()                                   # noqa: E731
    xr, ar, br = f(x), f(wgu), f(wdn)
    g, u = (xr @ ar.t()).chunk(2, 1)
    yr = (torch.nn.functional.silu(g) * u) @ br.t()
    yr.backward(dy.cpu().double())
    for name, got, ref in (("y", y, yr.detach()), ("dx", dx, xr.grad), ("dwgu", dwgu, ar.grad), ("dwdn", dwdn, br.grad)):
        rel = float((got.cpu().double() - ref).norm() / ref.norm())
        # a code's error is uniform in half a step: sigma = amax / (127 sqrt(12)), about 0.9 % of a Gaussian row's own
        # sigma (amax under 4 sigma); no result has more than eight such factors in all
        assert rel < 8 * 0.01, (name, rel)


@pytest.mark.parametrize("m", [70, 1100])
def test_block_step_captured_and_replayed(m):
    """The step in a graph, replayed with new inputs, eager work and
    synchronizations between: the bits of the eager step each time."""
    import quantized_gemm_int4_amd as hm
    d, k = 256, 384
    buf = _block_inputs(m, d, k, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            _block(hm, *buf)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _block(hm, *buf)
    for seed in range(1, 5):
        new = _block_inputs(m, d, k, seed)
        want = [t.clone() for t in _block(hm, *new)]
        for b, v in zip(buf, new):
            b.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(out, want):
            assert torch.equal(got, ref)


@pytest.mark.parametrize("m", [90, 1100])
def test_two_streams_and_repeated_calls(m):
    """Calls on two streams at once, and the same call again, give equal bits."""
    import quantized_gemm_int4_amd as hm
    ins = [_block_inputs(m, 256, 256, s) for s in (1, 2)]
    want = [[t.clone() for t in _block(hm, *i)] for i in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, i in zip(streams, ins):
            with torch.cuda.stream(s):
                got.append(_block(hm, *i))
    torch.cuda.synchronize()
    for j, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[j % 2]))


def test_stream_argument():
    import quantized_gemm_int4_amd as hm
    a = _dev(_layer(np.random.default_rng(1), 20, 64, 128))
    want = hm.hm_gemm_int8(*a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = hm.hm_gemm_int8(*a, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(ValueError):                            # shapes that do not belong together
        hm.hm_gemm_int8(a[0], a[1][:-1], a[2], a[3])
    with pytest.raises(ValueError):
        hm.hm_gemm_int8(a[0], a[1], a[2][:, :-1], a[3])
    with pytest.raises(ValueError):
        hm.hm_gemm_int8(a[0].t().contiguous().t(), a[1], a[2], a[3])
