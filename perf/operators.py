"""Operators beside the low-bit linear layer and around the MoE grouped GEMMs, as cases that can be timed:

* ``lora``, ``lora_grad``: low-rank adapters of many requests at once beside a shared projection, and their gradient;
* ``moe_dispatch``, ``moe_dispatch_grad``: token rows brought into expert order, and the gradient of that;
* ``moe_collect``, ``moe_collect_grad``: expert-ordered rows brought back to their tokens with the routing weights
  applied, and the gradient to the rows and to the weights.

With ``own`` false, ``run`` computes each operator in its plain form from elementary torch operations in fp32,
rounded once at the end; with ``own`` true it calls the library.  ``exact`` gives the definition in fp64.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
# Layers: n x k of the dense W4A16 layer (14336 x 4096), of the dense MXFP4 layer (7168 x 2048) and of the MoE
# gate_up projection (4096 x 7168); 256 experts, top-8, hidden 7168.


def listed():
    return [
        # one request decoding against its adapter: the smallest call, latency is all of it
        dict(name="lora_decode_one", kind="lora", m=1, n=7168, k=2048, rank=16, adapters=8, used=1, runs=False, none=0, keep_h=False),
        # a decode batch: 48 requests on 24 of 64 loaded adapters, some requests on the bare model
        dict(name="lora_decode_batch", kind="lora", m=48, n=14336, k=4096, rank=16, adapters=64, used=24, runs=False, none=5, keep_h=False),
        # a mixed step: prompts of a few requests, ragged, one adapter each; odd row and column counts
        dict(name="lora_mixed_ragged", kind="lora", m=1021, n=4099, k=7168, rank=64, adapters=16, used=7, runs=True, none=90, keep_h=False),
        # the forward pass of adapter training, several tenants' sequences in one batch, h kept for the gradient
        dict(name="lora_train_8192", kind="lora", m=8192, n=14336, k=4096, rank=64, adapters=6, used=6, runs=True, none=0, keep_h=True),
        # gradients of a small ragged training batch
        dict(name="lora_grad_ragged", kind="lora_grad", m=777, n=7168, k=2048, rank=16, adapters=4, used=3, runs=True, none=40),
        # gradients of one adapter over a full batch
        dict(name="lora_grad_8192", kind="lora_grad", m=8192, n=14336, k=4096, rank=32, adapters=1, used=1, runs=True, none=0),
        # a decode step's tokens to their experts
        dict(name="dispatch_decode_64", kind="moe_dispatch", t=64, topk=8, experts=256, local=256, n=7168),
        # a prefill or training batch's tokens to their experts
        dict(name="dispatch_8192", kind="moe_dispatch", t=8192, topk=8, experts=256, local=256, n=7168),
        # the gradient of a dispatch on a rank that holds a quarter of the experts: most pairs dropped, odd sizes
        dict(name="dispatch_grad_local", kind="moe_dispatch_grad", t=1003, topk=8, experts=256, local=64, n=2049),
        # a decode step's expert outputs back to its tokens
        dict(name="collect_decode_64", kind="moe_collect", t=64, topk=8, experts=256, local=256, n=7168),
        # gradients of the weighted sum: a small batch with two experts a token, and a large one
        dict(name="collect_grad_257", kind="moe_collect_grad", t=257, topk=2, experts=16, local=16, n=2048),
        dict(name="collect_grad_4096", kind="moe_collect_grad", t=4096, topk=8, experts=256, local=256, n=7168),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: decode to training lengths, every rank the adapters may have, one to 512 experts."""
    kind = rng.choice(["lora", "lora", "lora_grad", "moe_dispatch", "moe_dispatch_grad", "moe_collect", "moe_collect_grad"])
    if kind.startswith("lora"):
        k = 128 * _log(rng, 4, 56)
        n = _log(rng, 512, 14336)
        n = n if rng.random() < 0.3 else 16 * (n // 16)
        rank = rng.choice([8, 16, 16, 24, 32, 48, 64, 128])
        m = _log(rng, 1, 8192) if kind == "lora" else _log(rng, 16, 8192)
        adapters = _log(rng, 1, 64)
        used = min(adapters, max(1, m // 2), _log(rng, 1, 64))
        runs = m > 256 or rng.random() < 0.3
        none = min(m - used, rng.choice([0, 0, m // 10, m // 2]))
        c = dict(kind=kind, m=m, n=n, k=k, rank=rank, adapters=adapters, used=used, runs=runs, none=max(0, none))
        if kind == "lora":
            c["keep_h"] = rng.random() < 0.5
        return c
    experts = rng.choice([8, 16, 60, 64, 128, 256, 512])
    topk = rng.choice([1, 2, 3, 4, 6, 8, 8])
    n = _log(rng, 256, 7168)
    n = n if rng.random() < 0.2 else 8 * (n // 8)
    local = experts if rng.random() < 0.6 else max(topk, experts // rng.choice([2, 4, 8]))
    return dict(kind=kind, t=_log(rng, 1, 8192 if kind == "moe_dispatch" else 4096), topk=topk, experts=experts, local=local, n=n)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


def _adapter_ids(case, seed):
    """Adapter of every row, on the host: every used adapter at least once, the rest by popularity, in single rows
    (decode) or in runs (prompts); `none` rows have no adapter (-1)."""
    g = torch.Generator()
    g.manual_seed(int(seed) + 17)
    m, used = case["m"], case["used"]
    names = torch.randperm(case["adapters"], generator=g)[:used].to(torch.int32)
    busy = m - case["none"]
    p = 1.0 / (1.0 + torch.arange(used, dtype=torch.float64))
    if case["runs"]:
        # ragged runs: cut points at random, one adapter a run, as many runs as used adapters and half as many again
        nruns = min(busy, used + used // 2)
        cuts = torch.sort(torch.randperm(busy - 1, generator=g)[:nruns - 1] + 1).values if nruns > 1 else torch.zeros(0, dtype=torch.int64)
        lens = torch.diff(torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([busy])]))
        which = torch.cat([torch.arange(used), torch.randint(0, used, (nruns - used,), generator=g)])
        which = which[torch.randperm(nruns, generator=g)]
        ids = torch.cat([names[which].repeat_interleave(lens), torch.full((case["none"],), -1, dtype=torch.int32)])
    else:
        rest = torch.multinomial(p / p.sum(), busy - used, replacement=True, generator=g) if busy > used else torch.zeros(0, dtype=torch.int64)
        which = torch.cat([torch.arange(used), rest])
        ids = torch.cat([names[which], torch.full((case["none"],), -1, dtype=torch.int32)])
        ids = ids[torch.randperm(m, generator=g)]
    return ids


def _lora_inputs(case, seed):
    g = _gen(seed)
    m, n, k, r, L = (case[x] for x in ("m", "n", "k", "rank", "adapters"))
    ids = _adapter_ids(case, seed)
    s = dict(kind=case["kind"], ids=ids.cuda(), m=m, n=n, k=k, rank=r, adapters=L)
    # which rows an adapter has is known to the program that scheduled the batch
    s["rows"] = [(a, torch.nonzero(ids == a).flatten().cuda()) for a in torch.unique(ids[ids >= 0]).tolist()]
    s["single"] = not case["runs"] and m * r * (k + n) <= 1 << 28      # one row a request: the plain form gathers the adapters per row
    s["x"] = _randn(g, m, k)
    s["a"] = _randn(g, L, r, k, std=k ** -0.5)
    s["b"] = _randn(g, L, n, r, std=0.02)
    s["scales"] = torch.rand(L, generator=g, device="cuda") + 0.5
    if case["kind"] == "lora":
        s["base"] = _randn(g, m, n)
        s["keep_h"] = case["keep_h"]
    else:
        s["dy"] = _randn(g, m, n, std=0.05)
        s["dx_base"] = _randn(g, m, k, std=0.05)
        # the forward pass kept h = scale * A x: unit normal times the adapter's scale, 0 where there is none
        sc = torch.where(s["ids"] >= 0, s["scales"][s["ids"].clamp(min=0).long()], torch.zeros((), device="cuda"))
        s["h"] = torch.randn(m, r, generator=g, device="cuda") * sc[:, None]
    return s


def _route(g, t, topk, experts, local):
    """Top-k experts of Gaussian logits with a Zipf(1.1) popularity; experts held by other ranks become -1."""
    rank = torch.randperm(experts, generator=g, device="cuda").float()
    logits = torch.randn(t, experts, generator=g, device="cuda") - 1.1 * torch.log1p(rank)
    v, ids = torch.topk(logits, topk, dim=1)
    ids = torch.where(ids < local, ids, torch.full_like(ids, -1)).to(torch.int32).contiguous()
    return ids, torch.softmax(v, dim=1).contiguous()


def _plain_sort(ids, local):
    """counts, offsets, sorted pairs (dropped pairs behind the last, ascending) and each pair's position (-1: dropped)."""
    flat = ids.reshape(-1).long()
    ok = (flat >= 0) & (flat < local)
    key = torch.where(ok, flat, torch.full_like(flat, local))
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(local + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))[:local]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=ids.device), torch.cumsum(counts, 0)])
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=ids.device)
    pos = torch.where(ok, pos, torch.full_like(pos, -1))
    return counts, offsets, order, pos


def _moe_inputs(case, seed):
    g = _gen(seed)
    t, topk, n, local = case["t"], case["topk"], case["n"], case["local"]
    ids, w = _route(g, t, topk, case["experts"], local)
    s = dict(kind=case["kind"], ids=ids, local=local, t=t, topk=topk, n=n)
    if case["kind"] == "moe_dispatch":
        s["x"] = _randn(g, t, n)
        return s
    s["pos"] = _plain_sort(ids, local)[3].to(torch.int32).reshape(t, topk).contiguous()
    s["rows"] = _randn(g, t * topk, n)                 # expert outputs (collect) or their gradient's rows (dispatch)
    if case["kind"] != "moe_dispatch_grad":
        s["w"] = w
    if case["kind"] == "moe_collect_grad":
        s["dout"] = _randn(g, t, n)
    return s


def _inputs(case, seed):
    return _lora_inputs(case, seed) if case["kind"].startswith("lora") else _moe_inputs(case, seed)


def prepare(case, seed):
    """Inputs, and the output and workspace buffers that a serving or training loop keeps."""
    s = _inputs(case, seed)
    e = lambda *shape, dt=BF16: torch.empty(shape, dtype=dt, device="cuda")          # noqa: E731
    i32 = torch.int32
    kind = s["kind"]
    if kind == "lora":
        s["out"] = dict(y=e(s["m"], s["n"]))
        if s["keep_h"]:
            s["out"]["h"] = e(s["m"], s["rank"], dt=torch.float32)
    elif kind == "lora_grad":
        s["out"] = dict(dx=e(s["m"], s["k"]), da=e(s["adapters"], s["rank"], s["k"]), db=e(s["adapters"], s["n"], s["rank"]))
    elif kind == "moe_dispatch":
        P = s["t"] * s["topk"]
        # rows and pair ids behind the last routed pair are left as they are
        s["out"] = dict(xs=torch.zeros(P, s["n"], dtype=BF16, device="cuda"), counts=e(s["local"], dt=i32),
                        offsets=e(s["local"] + 1, dt=i32), sorted_pairs=torch.full((P,), -1, dtype=i32, device="cuda"),
                        positions=e(s["t"], s["topk"], dt=i32))
    elif kind == "moe_collect_grad":
        s["out"] = dict(dys=torch.zeros(s["t"] * s["topk"], s["n"], dtype=BF16, device="cuda"),
                        dweights=e(s["t"], s["topk"], dt=torch.float32))
    else:
        s["out"] = {("out" if kind == "moe_collect" else "dx"): e(s["t"], s["n"])}
    if own:
        import quantized_gemm_int4_amd as hm
        ws = 0
        if kind.startswith("lora"):
            s["desc"] = hm.lora_desc(s["n"], s["k"], s["rank"], s["adapters"])
            ws = (hm.hm_lora_workspace_size if kind == "lora" else hm.hm_lora_grad_workspace_size)(s["desc"], s["m"])
        elif kind == "moe_dispatch":
            ws = hm.hm_moe_dispatch_workspace_size(s["t"], s["topk"], s["local"])
        s["ws"] = torch.empty(max(ws, 256), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _PLAIN[s["kind"]](s)


def _run_own(s):
    import quantized_gemm_int4_amd as hm
    o, kind = s["out"], s["kind"]
    if kind == "lora":
        hm.hm_lora(s["desc"], s["x"], s["ids"], s["a"], s["b"], s["scales"], base=s["base"], y=o["y"], h=o.get("h"), ws=s["ws"])
    elif kind == "lora_grad":
        hm.hm_lora_grad(s["desc"], s["dy"], s["x"], s["h"], s["ids"], s["a"], s["b"], s["scales"], dx_base=s["dx_base"],
                        dx=o["dx"], da=o["da"], db=o["db"], ws=s["ws"])
    elif kind == "moe_dispatch":
        hm.hm_moe_dispatch(s["x"], s["ids"], s["local"], ws=s["ws"], **o)
    elif kind == "moe_dispatch_grad":
        hm.hm_moe_dispatch_grad(s["rows"], s["pos"], dx=o["dx"])
    elif kind == "moe_collect":
        hm.hm_moe_collect(s["rows"], s["w"], s["pos"], out=o["out"])
    else:
        hm.hm_moe_collect_grad(s["dout"], s["rows"], s["w"], s["pos"], **o)
    return o


def _plain_lora(s):
    x, base = s["x"].float(), s["base"].float()
    if s["single"]:
        ok = (s["ids"] >= 0)[:, None]
        i = s["ids"].clamp(min=0).long()
        h = (s["a"][i].float() @ x[:, :, None])[:, :, 0] * s["scales"][i][:, None] * ok
        y = base + (s["b"][i].float() @ h[:, :, None])[:, :, 0]
    else:
        y, h = base.clone(), torch.zeros(s["m"], s["rank"], device=x.device)
        for a, rows in s["rows"]:
            ha = (x[rows] @ s["a"][a].float().t()) * s["scales"][a]
            h[rows] = ha
            y[rows] += ha @ s["b"][a].float().t()
    o = dict(y=y.to(BF16))
    if s["keep_h"]:
        o["h"] = h
    return o


def _plain_lora_grad(s):
    dy, x, h = s["dy"].float(), s["x"].float(), s["h"]
    dx = s["dx_base"].float().clone()
    da = torch.zeros(s["a"].shape, device=x.device)
    db = torch.zeros(s["b"].shape, device=x.device)
    for a, rows in s["rows"]:
        dya = dy[rows]
        g = (dya @ s["b"][a].float()) * s["scales"][a]
        dx[rows] += g @ s["a"][a].float()
        da[a] = g.t() @ x[rows]
        db[a] = dya.t() @ h[rows]
    return dict(dx=dx.to(BF16), da=da.to(BF16), db=db.to(BF16))


def _plain_dispatch(s):
    counts, offsets, order, pos = _plain_sort(s["ids"], s["local"])
    behind = torch.arange(order.numel(), device=order.device) >= offsets[-1]
    xs = torch.where(behind[:, None], torch.zeros((), dtype=BF16, device=order.device), s["x"][order // s["topk"]])
    i32 = torch.int32
    return dict(xs=xs, counts=counts.to(i32), offsets=offsets.to(i32),
                sorted_pairs=torch.where(behind, torch.full_like(order, -1), order).to(i32), positions=pos.to(i32).reshape(s["ids"].shape))


def _plain_sum(s):
    t, topk, n = s["t"], s["topk"], s["n"]
    acc = torch.zeros(t, n, device=s["rows"].device)
    for j in range(topk):
        p = s["pos"][:, j].long()
        v = s["rows"][p.clamp(min=0)].float()
        if "w" in s:
            v = v * s["w"][:, j:j + 1]
        acc += torch.where((p >= 0)[:, None], v, torch.zeros((), device=v.device))
    return {("out" if "w" in s else "dx"): acc.to(BF16)}


def _plain_collect_grad(s):
    t, topk, n = s["t"], s["topk"], s["n"]
    dys = torch.zeros(t * topk + 1, n, dtype=BF16, device=s["rows"].device)       # the last row takes the dropped pairs
    dw = torch.empty(t, topk, device=dys.device)
    dout = s["dout"].float()
    for j in range(topk):
        p = s["pos"][:, j].long()
        dw[:, j] = torch.where(p >= 0, (dout * s["rows"][p.clamp(min=0)].float()).sum(1), torch.zeros((), device=dys.device))
        dys[torch.where(p >= 0, p, torch.full_like(p, t * topk))] = (dout * s["w"][:, j:j + 1]).to(BF16)
    return dict(dys=dys[:-1], dweights=dw)


_PLAIN = dict(lora=_plain_lora, lora_grad=_plain_lora_grad, moe_dispatch=_plain_dispatch, moe_dispatch_grad=_plain_sum,
              moe_collect=_plain_sum, moe_collect_grad=_plain_collect_grad)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    f = torch.float64
    kind = s["kind"]
    if kind.startswith("lora"):
        m, ids = s["m"], s["ids"].long()
        x, A, B = s["x"].to(f), s["a"], s["b"]
        if kind == "lora":
            y, h = s["base"].to(f), torch.zeros(m, s["rank"], dtype=f, device=x.device)
        else:
            dx, dy, h = s["dx_base"].to(f), s["dy"].to(f), s["h"].to(f)
            da, db = torch.zeros(A.shape, dtype=f, device=x.device), torch.zeros(B.shape, dtype=f, device=x.device)
        for a in range(s["adapters"]):
            r = (ids == a).nonzero()[:, 0]
            if r.numel() == 0:
                continue
            sc, Aa, Ba = s["scales"][a].to(f), A[a].to(f), B[a].to(f)
            if kind == "lora":
                h[r] = sc * torch.mm(x[r], Aa.t())
                y[r] = y[r] + torch.mm(h[r], Ba.t())
            else:
                gr = sc * torch.mm(dy[r], Ba)
                dx[r] = dx[r] + torch.mm(gr, Aa)
                da[a] = torch.mm(gr.t(), x[r])
                db[a] = torch.mm(dy[r].t(), h[r])
        if kind == "lora_grad":
            return dict(dx=dx, da=da, db=db)
        return dict(y=y, h=h) if s["keep_h"] else dict(y=y)
    if kind == "moe_dispatch":
        # copies, and whole numbers that are equal or wrong
        flat, P = s["ids"].reshape(-1), s["t"] * s["topk"]
        pairs = torch.cat([torch.nonzero(flat == e)[:, 0] for e in range(s["local"])])
        xs = torch.zeros(P, s["n"], dtype=f, device=flat.device)
        xs[:pairs.numel()] = s["x"][torch.div(pairs, s["topk"], rounding_mode="floor")].to(f)
        return dict(xs=xs, counts=None, offsets=None, sorted_pairs=None, positions=None)
    t, topk, n = s["t"], s["topk"], s["n"]
    pos = s["pos"].long().reshape(-1)
    pair = torch.nonzero(pos >= 0)[:, 0]
    tok = pair // topk
    if kind == "moe_collect_grad":
        dys = torch.zeros(t * topk, n, dtype=f, device=pos.device)
        dw = torch.zeros(t * topk, dtype=f, device=pos.device)
        dys[pos[pair]] = s["w"].to(f).reshape(-1)[pair][:, None] * s["dout"].to(f)[tok]
        for lo in range(0, pair.numel(), 4096):
            q = pair[lo:lo + 4096]
            dw[q] = (s["dout"][q // topk].to(f) * s["rows"][pos[q]].to(f)).sum(1)
        return dict(dys=dys, dweights=dw.reshape(t, topk))
    out = torch.zeros(t, n, dtype=f, device=pos.device)
    v = s["rows"].to(f)[pos[pair]]
    if kind == "moe_collect":
        v = v * s["w"].to(f).reshape(-1)[pair][:, None]
    out.index_add_(0, tok, v)
    return {("out" if kind == "moe_collect" else "dx"): out}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    kind = case["kind"]
    if kind.startswith("lora"):
        m, n, k, r, L, used = (case[x] for x in ("m", "n", "k", "rank", "adapters", "used"))
        busy = m - case["none"]
        if kind == "lora":
            # x and the used adapters in; base in, y out; h out where it is kept
            nb = 2 * busy * k + 2 * used * r * (k + n) + 4 * m * n + 4 * m + 4 * used + (4 * m * r if case["keep_h"] else 0)
            return dict(bytes=nb, flops=2 * busy * r * (k + n))
        # dy, x, h and the used adapters in; dx_base in, dx out; da and db out for every adapter
        nb = 2 * busy * (n + k) + 4 * busy * r + 4 * m * k + 2 * used * r * (k + n) + 2 * L * r * (k + n) + 4 * m
        return dict(bytes=nb, flops=4 * busy * r * (k + n))
    t, topk, n, E = case["t"], case["topk"], case["n"], case["local"]
    P = t * topk
    # experts kept of all: the share of pairs that stay (popular experts are spread at random over the ranks)
    live = int(round(P * min(1.0, E / case["experts"])))
    if kind == "moe_dispatch":
        # ids and x in; the rows, pair ids and positions, counts and offsets out
        return dict(bytes=2 * t * n + 2 * live * n + 12 * P + 8 * E, flops=0)
    if kind == "moe_collect_grad":
        return dict(bytes=2 * t * n + 4 * live * n + 12 * P, flops=3 * live * n)
    return dict(bytes=2 * t * n + 2 * live * n + (8 if kind == "moe_collect" else 4) * P, flops=(2 if kind == "moe_collect" else 1) * live * n)
