"""Pins of the oracle's low-rank adapters and of its expert-order rows: hand
values, a dense weight update as the second way to the same result, and the
gradients against central differences in float64."""
import numpy as np
import pytest

from oracle import lora, moe


def test_lora_hand_values():
    x = np.array([[1.0, 2.0], [3.0, -1.0], [5.0, 5.0]])
    a = np.array([[[1.0, 0.0]], [[0.5, 1.0]]])              # L = 2, rank 1, K = 2
    b = np.array([[[2.0], [0.0]], [[1.0], [-1.0]]])         # N = 2
    (y, h), _ = lora.lora_ref(x, [0, 1, -1], a, b, [10.0, 2.0], base=np.ones((3, 2)))
    assert np.array_equal(h, [[10.0], [1.0], [0.0]])        # 10*1; 2*(1.5-1); none
    assert np.array_equal(y, [[21.0, 1.0], [2.0, 0.0], [1.0, 1.0]])


@pytest.mark.parametrize("seed", range(3))
def test_lora_equals_dense_update(seed):
    r = np.random.default_rng(seed)
    M, K, N, R, L = 9, 12, 7, 4, 3
    x, a, b = r.normal(size=(M, K)), r.normal(size=(L, R, K)), r.normal(size=(L, N, R))
    s, ids, base = r.normal(size=L), r.integers(-1, L + 1, M), r.normal(size=(M, N))
    (y, _), (by, _) = lora.lora_ref(x, ids, a, b, s, base)
    for m in range(M):
        w = s[ids[m]] * b[ids[m]] @ a[ids[m]] if 0 <= ids[m] < L else np.zeros((N, K))
        assert np.allclose(y[m], base[m] + w @ x[m], atol=1e-12)
    assert (by >= np.abs(y) - 1e-12).all()


def test_lora_gradient_against_differences():
    r = np.random.default_rng(5)
    M, K, N, R, L = 6, 5, 4, 3, 3
    x, a, b = r.normal(size=(M, K)), r.normal(size=(L, R, K)), r.normal(size=(L, N, R))
    s, ids, dy = r.normal(size=L), np.array([0, 1, 1, -1, 0, 7]), r.normal(size=(M, N))
    loss = lambda: float((lora.lora_ref(x, ids, a, b, s)[0][0] * dy).sum())              # noqa: E731
    h = lora.lora_ref(x, ids, a, b, s)[0][1]
    grads = lora.lora_grad_ref(dy, x, h, ids, a, b, s)[0]
    for v, g in zip((x, a, b), grads):
        f, gf = v.reshape(-1), g.reshape(-1)
        for i in range(f.size):
            keep = f[i]
            f[i] = keep + 1e-5
            up = loss()
            f[i] = keep - 1e-5
            down = loss()
            f[i] = keep
            # the loss is cubic at most: the difference's error is 1e-10 times a third derivative, and rounding 1e-11
            assert abs((up - down) / 2e-5 - gf[i]) < 1e-8
    assert (grads[1][2] == 0).all() and (grads[2][2] == 0).all()       # no row uses adapter 2


def test_positions_hand_and_against_sort():
    pos, off = moe.positions_ref(np.array([[2, 0], [0, -1], [5, 2]]), 3)
    assert pos.tolist() == [[2, 0], [1, -1], [-1, 3]] and off.tolist() == [0, 2, 2, 4]
    ids = np.random.default_rng(0).integers(0, 9, (40, 3))
    pos, off = moe.positions_ref(ids, 9)
    _, ro, sp = moe.moe_sort_ref(ids, 9)
    assert np.array_equal(off, ro) and np.array_equal(pos.ravel()[sp], np.arange(120))


def test_collect_gradient_against_differences():
    r = np.random.default_rng(8)
    t, topk, n = 4, 3, 5
    pos, _ = moe.positions_ref(r.integers(-1, 3, (t, topk)), 3)
    ys, w, dout = r.normal(size=(t * topk, n)), r.normal(size=(t, topk)), r.normal(size=(t, n))
    dys, dw, _ = moe.collect_grad_ref(dout, ys, w, pos)
    dys = np.nan_to_num(dys)
    for v, g in ((ys, dys), (w, dw)):
        f, gf = v.reshape(-1), g.reshape(-1)
        for i in range(f.size):
            keep = f[i]
            f[i] = keep + 0.5
            up = (moe.collect_ref(ys, w, pos)[0] * dout).sum()
            f[i] = keep - 0.5
            down = (moe.collect_ref(ys, w, pos)[0] * dout).sum()
            f[i] = keep
            assert abs((up - down) - gf[i]) < 1e-10                     # linear in each: exact but for rounding
