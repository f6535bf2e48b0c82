"""Linear layers in 8-bit integers, with one scale for each token and each output channel, as cases that can be timed:

* ``quant``: bf16 rows to int8 codes and a scale a row (what the product reads, and what a training step keeps of its activations);
* ``gemm``: the product of such rows with such weights;
* ``gated``: the gate and up projections of a feed-forward block with SiLU and the product, in one call;
* ``gated_grad``: the gradient of that to gate and up, computed again from the 8-bit rows;
* ``grad``: the gradient of the product to its rows and to its weights, from the 8-bit rows and weights.

With ``own`` false, ``run`` computes each operator in its plain form from elementary torch operations in fp32,
rounded once at the end; with ``own`` true it calls the library.  ``exact`` gives the definition in fp64.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
# Layers: n x k of the dense W4A16 layer (14336 x 4096), of the dense MXFP4 layer (7168 x 2048) and of the MoE
# gate_up projection (4096 x 7168).


def listed():
    return [
        # a decode batch's rows before a projection: the smallest call, latency is all of it
        dict(name="quant_decode_48", kind="quant", m=48, k=4096),
        # a training batch's feed-forward activations, kept in 8 bits for the backward pass
        dict(name="quant_train_8192", kind="quant", m=8192, k=14336),
        # one request decoding: the weights are read once and that is all
        dict(name="gemm_decode_one", kind="gemm", m=1, n=14336, k=4096),
        # a decode batch on a narrower layer
        dict(name="gemm_decode_48", kind="gemm", m=48, n=7168, k=2048),
        # a mixed step of prompts and decoding requests, ragged; an odd number of columns
        dict(name="gemm_mixed_1021", kind="gemm", m=1021, n=4099, k=7168),
        # a prefill or training batch
        dict(name="gemm_train_8192", kind="gemm", m=8192, n=14336, k=4096),
        # the feed-forward block's first half for a small decode batch
        dict(name="gated_decode_4", kind="gated", m=4, d=7168, k=2048),
        # and for a training batch
        dict(name="gated_train_4096", kind="gated", m=4096, d=14336, k=4096),
        # its gradient in a small ragged training batch (a shard of 2049 columns)
        dict(name="gated_grad_777", kind="gated_grad", m=777, d=2049, k=7168),
        # and over a whole one
        dict(name="gated_grad_4096", kind="gated_grad", m=4096, d=14336, k=4096),
        # gradients of a projection in a small ragged batch
        dict(name="grad_333", kind="grad", m=333, n=7168, k=2048),
        # and over a whole one
        dict(name="grad_4096", kind="grad", m=4096, n=14336, k=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: one token to a training batch, narrow and wide layers, odd numbers of rows and columns."""
    kind = rng.choice(["quant", "gemm", "gemm", "gated", "gated_grad", "grad"])
    if kind == "quant":
        k = _log(rng, 128, 14336)
        return dict(kind=kind, m=_log(rng, 1, 8192), k=k if rng.random() < 0.3 else 128 * max(1, k // 128))
    k = 128 * _log(rng, 2, 56)
    n = _log(rng, 256, 14336)
    n = n if rng.random() < 0.3 else 64 * (n // 64)
    # rows up to a training batch, as many as keep the pass under the largest listed one
    m = _log(rng, 1 if kind in ("gemm", "gated") else 16, 8192 if kind == "gemm" else 4096)
    m = min(m, (8192 if kind == "gemm" else 4096) * 14336 * 4096 // (n * k))
    return dict(kind=kind, m=m, k=k, **({"n": n} if kind in ("gemm", "grad") else {"d": n}))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, m, k):
    """Unit normal rows with a few channels that are much larger than the others, as transformer activations have."""
    x = torch.randn(m, k, generator=g, device="cuda")
    big = torch.randint(0, k, (max(1, k // 512),), generator=g, device="cuda")
    x[:, big] *= 8.0
    return x.to(BF16)


def _to_int8(x):
    """Codes and fp32 scales of rows: s = amax / 127, the code the nearest whole number to 127 x / amax, ties to even.
    The division is in fp64, where every tie is met exactly."""
    amax = x.abs().amax(1, keepdim=True)
    scale = (amax.float() / 127.0)[:, 0]
    q = torch.where(amax > 0, torch.round(x.double() * 127.0 / amax.double()), torch.zeros((), dtype=torch.float64, device=x.device))
    return q.to(torch.int8), scale


def _inputs(case, seed):
    g = _gen(seed)
    kind, m, k = case["kind"], case["m"], case["k"]
    s = dict(kind=kind, m=m, k=k)
    x = _activations(g, m, k)
    if kind == "quant":
        s["x"] = x
        return s
    s["x8"], s["sx"] = _to_int8(x)
    s["n"] = n = case["n"] if "n" in case else 2 * case["d"]       # rows of the weights: gate rows, then up rows
    # the scale of a channel belongs to its weights, fp32
    s["w8"], s["sw"] = _to_int8(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5)
    if kind == "gated_grad":
        s["dh"] = (torch.randn(m, n // 2, generator=g, device="cuda") * 0.05).to(BF16)
    if kind == "grad":
        s["dy"] = (torch.randn(m, n, generator=g, device="cuda") * 0.05).to(BF16)
    return s


def prepare(case, seed):
    """Inputs, and the output and workspace buffers that a serving or training loop keeps."""
    s = _inputs(case, seed)
    kind, m, k = s["kind"], s["m"], s["k"]
    e = lambda *shape, dt=BF16: torch.empty(shape, dtype=dt, device="cuda")          # noqa: E731
    if kind == "quant":
        s["out"] = dict(x8=e(m, k, dt=torch.int8), row_scale=e(m, dt=torch.float32))
        return s
    n = s["n"]
    s["out"] = {"gemm": lambda: dict(y=e(m, n)), "gated": lambda: dict(h=e(m, n // 2)), "gated_grad": lambda: dict(dgu=e(m, n)),
                "grad": lambda: dict(dx=e(m, k), dw=e(n, k))}[kind]()
    if own:
        import quantized_gemm_int4_amd as hm
        size = {"gemm": hm.hm_gemm_int8_workspace_size, "gated": hm.hm_gemm_int8_gated_workspace_size,
                "gated_grad": hm.hm_gemm_int8_gated_grad_workspace_size, "grad": hm.hm_gemm_int8_grad_workspace_size}[kind]
        s["ws"] = torch.empty(max(size(m, n, k), 256), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _PLAIN[s["kind"]](s)


def _run_own(s):
    import quantized_gemm_int4_amd as hm
    o, kind = s["out"], s["kind"]
    if kind == "quant":
        hm.hm_quant_int8_rows(s["x"], **o)
        return o
    a = (s["x8"], s["sx"], s["w8"], s["sw"])
    if kind == "gemm":
        hm.hm_gemm_int8(*a, ws=s["ws"], **o)
    elif kind == "gated":
        hm.hm_gemm_int8_gated(*a, ws=s["ws"], **o)
    elif kind == "gated_grad":
        hm.hm_gemm_int8_gated_grad(s["dh"], *a, ws=s["ws"], **o)
    else:
        hm.hm_gemm_int8_grad(s["dy"], *a, ws=s["ws"], **o)
    return o


def _plain_quant(s):
    x8, scale = _to_int8(s["x"])
    return dict(x8=x8, row_scale=scale)


def _plain_product(s):
    return (s["x8"].float() @ s["w8"].float().t()) * s["sx"][:, None] * s["sw"]


def _plain_gemm(s):
    return dict(y=_plain_product(s).to(BF16))


def _plain_gated(s):
    g, u = _plain_product(s).chunk(2, 1)
    return dict(h=(g / (1.0 + torch.exp(-g)) * u).to(BF16))


def _plain_gated_grad(s):
    g, u = _plain_product(s).chunk(2, 1)
    dh = s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    return dict(dgu=torch.cat([dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig], 1).to(BF16))


def _plain_grad(s):
    dy = s["dy"].float()
    dx = dy @ (s["w8"].float() * s["sw"][:, None])
    dw = dy.t() @ (s["x8"].float() * s["sx"][:, None])
    return dict(dx=dx.to(BF16), dw=dw.to(BF16))


_PLAIN = dict(quant=_plain_quant, gemm=_plain_gemm, gated=_plain_gated, gated_grad=_plain_gated_grad, grad=_plain_grad)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    f = torch.float64
    kind = s["kind"]
    if kind == "quant":
        # codes are whole numbers, equal or wrong
        return dict(x8=None, row_scale=s["x"].to(f).abs().max(dim=1).values / 127)
    if kind == "grad":
        w_hat = s["w8"].to(f).mul_(s["sw"].to(f).unsqueeze(1))
        dx = torch.mm(s["dy"].to(f), w_hat)
        del w_hat
        x_hat = s["x8"].to(f).mul_(s["sx"].to(f).unsqueeze(1))
        return dict(dx=dx, dw=torch.mm(s["dy"].to(f).t(), x_hat))
    # whole numbers: the products of 512 codes sum to less than 2^24, exact in any order in fp32, and are summed in fp64
    out = []
    half = s["n"] // 2
    for lo in range(0, s["m"], 1024):
        rows = s["x8"][lo:lo + 1024]
        acc = torch.zeros(rows.shape[0], s["n"], dtype=f, device=rows.device)
        for c in range(0, s["k"], 512):
            acc += torch.mm(rows[:, c:c + 512].float(), s["w8"][:, c:c + 512].float().t())
        acc *= torch.outer(s["sx"][lo:lo + 1024].to(f), s["sw"].to(f))
        if kind == "gemm":
            out.append(acc)
            continue
        g, u = acc[:, :half], acc[:, half:]
        p = torch.sigmoid(g)
        if kind == "gated":
            out.append(g * p * u)
        else:
            dh = s["dh"][lo:lo + 1024].to(f)
            out.append(torch.cat([dh * u * (p + g * p * (1 - p)), dh * g * p], 1))
    return {{"gemm": "y", "gated": "h", "gated_grad": "dgu"}[kind]: torch.cat(out)}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    kind, m, k = case["kind"], case["m"], case["k"]
    if kind == "quant":
        # rows in; codes and scales out; absolute value, maximum and product
        return dict(bytes=3 * m * k + 4 * m, flops=3 * m * k)
    n = case["n"] if "n" in case else 2 * case["d"]
    codes = m * k + n * k + 4 * m + 4 * n
    if kind == "gemm":
        return dict(bytes=codes + 2 * m * n, flops=2 * m * n * k)
    if kind == "gated":
        return dict(bytes=codes + m * n, flops=2 * m * n * k)
    if kind == "gated_grad":
        # dh in, the gradients of gate and up out
        return dict(bytes=codes + m * n + 2 * m * n, flops=2 * m * n * k)
    # dy in once, dx and dw out
    return dict(bytes=codes + 2 * m * n + 2 * m * k + 2 * n * k, flops=4 * m * n * k)
