"""The oracle of the 8-bit integer layers against brute force: rational
arithmetic for the codes, differences for the gradients."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import codecs, int8


def _bf16(r, *shape, std=1.0):
    return codecs.bf16_value(codecs.bf16_rne_bits(r.normal(0, std, shape).astype(np.float32))).astype(np.float64)


def test_codes_are_the_nearest_of_the_exact_quotient():
    r = np.random.default_rng(3)
    x = np.concatenate([_bf16(r, 4, 300), np.arange(-150, 150)[None, :] * 1.0, np.zeros((1, 300))])
    x[0, :4] = [2.0, 1.0, -1.0, 0.5]
    x[4] = np.clip(x[4], -127, 127) * 2                      # amax 254: odd values are ties
    x[4, ::2] = np.arange(-127, 127, 254 / 150).round()[:150] * 1.0
    q, s = int8.quant_rows(x)
    for i in range(x.shape[0]):
        a = Fraction(float(np.abs(x[i]).max()))
        for j in range(x.shape[1]):
            if a == 0:
                assert q[i, j] == 0
                continue
            v = Fraction(float(x[i, j])) * 127 / a
            assert q[i, j] == round(v)                       # round() of a Fraction: ties to even
    assert s[-1] == 0 and np.array_equal(s, np.abs(x).max(1).astype(np.float32) / np.float32(127))


def test_rows_that_are_not_finite():
    x = np.ones((3, 8))
    x[0, 3], x[1, 2] = np.inf, np.nan
    q, s = int8.quant_rows(x)
    assert np.isnan(s[:2]).all() and not q[:2].any() and (q[2] == 127).all()


def _layer(r, m, n, k):
    return (r.integers(-128, 128, (m, k)), r.uniform(0.5, 2, m).astype(np.float32) / 500, r.integers(-128, 128, (n, k)),
            r.uniform(0.5, 2, n).astype(np.float32) / 500)


def test_product_by_hand():
    r = np.random.default_rng(5)
    qx, sx, qw, sw = _layer(r, 3, 5, 128)
    y = int8.product(qx, sx, qw, sw)
    for m in range(3):
        for n in range(5):
            want = float(sx[m]) * float(sw[n]) * sum(int(a) * int(b) for a, b in zip(qx[m], qw[n]))
            assert abs(y[m, n] - want) <= 1e-12 * abs(want) + 1e-15


@pytest.mark.parametrize("seed", range(3))
def test_gradients_against_differences(seed):
    r = np.random.default_rng(seed)
    m, d, k = 3, 4, 128
    qx, sx, qw, sw = _layer(r, m, 2 * d, k)
    dh = r.normal(size=(m, d))
    dg, du, g, u = int8.gated_grad(dh, qx, sx, qw, sw)
    f = lambda g, u: float((dh * g * int8.sigmoid(g) * u).sum())                     # noqa: E731
    e = 1e-6
    for i in range(m):
        for j in range(d):
            t = np.zeros_like(g)
            t[i, j] = e
            assert abs((f(g + t, u) - f(g - t, u)) / (2 * e) - dg[i, j]) < 1e-6
            assert abs((f(g, u + t) - f(g, u - t)) / (2 * e) - du[i, j]) < 1e-6
    dy = r.normal(size=(m, 2 * d))
    (dx, dw), _ = int8.grad(dy, qx, sx, qw, sw)
    xh, wh = qx * sx[:, None].astype(float), qw * sw[:, None].astype(float)
    loss = lambda x, w: float((dy * (x @ w.T)).sum())                                # noqa: E731
    for i, j in ((0, 0), (2, 127), (1, 64)):
        t = np.zeros_like(xh)
        t[i, j] = 1e-4
        assert abs((loss(xh + t, wh) - loss(xh - t, wh)) / 2e-4 - dx[i, j]) < 1e-6
        t = np.zeros_like(wh)
        t[i, j] = 1e-4
        assert abs((loss(xh, wh + t) - loss(xh, wh - t)) / 2e-4 - dw[i, j]) < 1e-6


def test_sigmoid_far_out():
    g = np.array([-2000.0, -50.0, 0.0, 50.0, 2000.0])
    assert np.allclose(int8.sigmoid(g), [0.0, np.exp(-50.0), 0.5, 1.0, 1.0])
