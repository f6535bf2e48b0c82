"""Low-rank adapter reference (oracle side), NumPy float64, one row at a time
in the order the definition states:

  h[m] = s_e A_e x[m],   y[m] = base[m] + B_e h[m],      e = ids[m]
  g[m] = s_e B_e^T dy[m], dx[m] = dx_base[m] + A_e^T g[m],
  dA_e = sum over the rows m of e of g[m] x[m]^T,  dB_e = sum of dy[m] h[m]^T

Rows whose id lies outside [0, L) have no adapter (h = 0, y = base, dx =
dx_base, nothing added to dA, dB).  The adapters sit beside one linear layer
(ywsung.com note "How vLLM Humming computes 4 bits", section on one token vs
many tokens: a layer is X times W transposed); the pages do not define them,
the formulas are the plainest reading of a low-rank update of that layer.

Every function also returns, next to each result, the sum of the absolute
values of its terms, which the error bounds are stated in.
"""
import numpy as np


def lora_ref(x, ids, a, b, scales, base=None):
    """(y, h), (bound_y, bound_h); x [M,K], a [L,r,K], b [L,N,r], base [M,N]."""
    x, a, b, scales = (np.asarray(v, dtype=np.float64) for v in (x, a, b, scales))
    M, L, r, N = x.shape[0], a.shape[0], a.shape[1], b.shape[1]
    y = np.zeros((M, N)) if base is None else np.array(base, dtype=np.float64)
    by = np.abs(y)
    h, bh = np.zeros((M, r)), np.zeros((M, r))
    for m in range(M):
        e = int(ids[m])
        if 0 <= e < L:
            h[m] = scales[e] * (a[e] @ x[m])
            bh[m] = abs(scales[e]) * (np.abs(a[e]) @ np.abs(x[m]))
            y[m] += b[e] @ h[m]
            by[m] += np.abs(b[e]) @ bh[m]
    return (y, h), (by, bh)


def lora_grad_ref(dy, x, h, ids, a, b, scales, dx_base=None):
    """(dx, da, db), (bound_dx, bound_da, bound_db)."""
    dy, x, h, a, b, scales = (np.asarray(v, dtype=np.float64) for v in (dy, x, h, a, b, scales))
    M, L = x.shape[0], a.shape[0]
    dx = np.zeros_like(x) if dx_base is None else np.array(dx_base, dtype=np.float64)
    bdx = np.abs(dx)
    da, db = np.zeros_like(a), np.zeros_like(b)
    bda, bdb = np.zeros_like(a), np.zeros_like(b)
    for m in range(M):
        e = int(ids[m])
        if 0 <= e < L:
            g = scales[e] * (dy[m] @ b[e])
            bg = abs(scales[e]) * (np.abs(dy[m]) @ np.abs(b[e]))
            dx[m] += g @ a[e]
            bdx[m] += bg @ np.abs(a[e])
            da[e] += np.outer(g, x[m])
            bda[e] += np.outer(bg, np.abs(x[m]))
            db[e] += np.outer(dy[m], h[m])
            bdb[e] += np.outer(np.abs(dy[m]), np.abs(h[m]))
    return (dx, da, db), (bdx, bda, bdb)
