"""Reference of the 8-bit integer layers (oracle side), NumPy float64 and whole
numbers, from the definitions:

  x_hat = s_x[m] q_x[m,k],  w_hat = s_w[n] q_w[n,k]          codes int8, scales fp32
  quantization of a row:  s = amax / 127 (fp32),  q = nearest whole number to
                          127 x / amax, ties to even
  product                 y = x_hat w_hat^T
  gated block             h = silu(g) u,  [g | u] = x_hat w_hat^T
  its gradient            dg = dh u s (1 + g (1 - s)),  du = dh g s,  s = 1 / (1 + e^-g)
  product's gradient      dx = dy w_hat,  dw = dy^T x_hat

W8A8 is among the GEMM types of the pages' format list (cocoloop.cn news item),
which give no formulas; these are the plainest reading of symmetric 8-bit codes
with per-token and per-channel scales.
"""
import numpy as np


def quant_rows(x):
    """x float64 [m, k] holding bf16 values -> (int8 codes, fp32 scales).  127 x
    is exact in float64 and a quotient that is a tie is exact too, so rint sees
    the ratio's own ties.  Rows with an infinity or NaN: scale NaN, codes 0."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(axis=1)
    a = np.where(bad, 1.0, np.abs(np.where(np.isfinite(x), x, 0.0)).max(axis=1))
    q = np.zeros(x.shape, dtype=np.int8)
    for i in range(x.shape[0]):
        if not bad[i] and a[i] > 0:
            q[i] = np.rint(127.0 * x[i] / a[i]).astype(np.int8)
    s = a.astype(np.float32) / np.float32(127.0)
    s[bad] = np.nan
    return q, s


def product(qx, sx, qw, sw):
    """fp64 [m, n]: the whole-number sum (exact) times both scales."""
    acc = np.asarray(qx, dtype=np.float64) @ np.asarray(qw, dtype=np.float64).T
    with np.errstate(invalid="ignore", over="ignore"):
        return acc * np.asarray(sx, dtype=np.float64)[:, None] * np.asarray(sw, dtype=np.float64)[None, :]


def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def gated(qx, sx, qw, sw):
    """(h, g, u) in fp64; rows of qw: gate, then up."""
    p = product(qx, sx, qw, sw)
    d = p.shape[1] // 2
    g, u = p[:, :d], p[:, d:]
    return g * sigmoid(g) * u, g, u


def gated_grad(dh, qx, sx, qw, sw):
    """(dg, du, g, u) in fp64."""
    _, g, u = gated(qx, sx, qw, sw)
    s, rest = sigmoid(g), sigmoid(-g)
    return dh * u * s * (1.0 + g * rest), dh * g * s, g, u


def grad(dy, qx, sx, qw, sw):
    """(dx, dw) and the sums of the absolute values of their terms."""
    xh = np.asarray(qx, dtype=np.float64) * np.asarray(sx, dtype=np.float64)[:, None]
    wh = np.asarray(qw, dtype=np.float64) * np.asarray(sw, dtype=np.float64)[:, None]
    dy = np.asarray(dy, dtype=np.float64)
    return (dy @ wh, dy.T @ xh), (np.abs(dy) @ np.abs(wh), np.abs(dy).T @ np.abs(xh))
