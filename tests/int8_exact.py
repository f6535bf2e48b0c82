"""Inputs of the int8 layers' gradients whose results have one right bit pattern,
whatever the order of the sums, and those results.

whole: dy of -1, 0 and 1, scales of 1/2, 1 and 2.  Every term is a whole number of halves, and the sum of all terms'
  magnitudes stays under 2^24 halves, so every partial sum is exact in fp32; the one rounding left is the result's.
  A term lost, counted twice or given a neighbour's scale moves results by many of their steps.
chosen: one value of dy in each row (for dx; in each column for dw), scales of any kind: a result is one product
  of two bf16 numbers, exact in fp32, and so shows the rounding of scale times code."""
import torch

BF16, F = torch.bfloat16, torch.float64


def _gen(device, seed):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return dict(generator=g, device=device)


def operand(q, s):
    """bf16(scale code), the factor that hm_gemm_int8_grad is defined with."""
    return (q.float() * s[:, None]).to(BF16)


def whole(m, n, k, device, seed):
    """dy and (x8, x_scales, w8, w_scales)."""
    one = _gen(device, seed)
    top = min(128, 2 ** 22 // max(m, n))                       # terms of at most 2 top, max(m, n) of them
    q = lambda r: torch.randint(-top, min(top, 127) + 1, (r, k), dtype=torch.int8, **one)       # noqa: E731
    s = lambda r: torch.exp2(torch.randint(-1, 2, (r,), **one).float())                         # noqa: E731
    dy = torch.randint(-1, 2, (m, n), dtype=torch.int8, **one).to(BF16)
    return dy, (q(m), s(m), q(n), s(n))


def whole_results(dy, a, rows, cols):
    """Rows `rows` of dx and `cols` of dw: sums exact in 64 bits, rounded once (float() is exact under 2^24 halves)."""
    x, w = operand(a[0], a[1]).to(F), operand(a[2], a[3]).to(F)
    dx = dy[rows].to(F) @ w
    dw = dy[:, cols].t().contiguous().to(F) @ x
    return dx.float().to(BF16), dw.float().to(BF16)


def chosen(m, n, k, device, seed):
    """(dy for dx, its columns and values), (dy for dw, its rows and values), (x8, x_scales, w8, w_scales)."""
    one = _gen(device, seed)
    q = lambda r: torch.randint(-128, 128, (r, k), dtype=torch.int8, **one)                     # noqa: E731
    s = lambda r: torch.rand(r, **one) + 0.01                                                   # noqa: E731
    v = lambda r: torch.randn(r, **one).to(BF16)                                                # noqa: E731
    a = (q(m), s(m), q(n), s(n))
    col, row, vx, vw = torch.randint(0, n, (m,), **one), torch.randint(0, m, (n,), **one), v(m), v(n)
    col[-1], row[-1] = n - 1, m - 1                            # the last term of all is among them
    dyx, dyw = torch.zeros(m, n, dtype=BF16, device=device), torch.zeros(m, n, dtype=BF16, device=device)
    dyx[torch.arange(m, device=device), col] = vx
    dyw[row, torch.arange(n, device=device)] = vw
    return (dyx, col, vx), (dyw, row, vw), a


def chosen_result(of, values, q, s):
    """The result rows: values[i] times row of[i] of the operand (a product of two 8-bit significands is exact in fp32)."""
    return (values.float()[:, None] * operand(q[of], s[of]).float()).to(BF16)
