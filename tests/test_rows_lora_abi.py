"""Argument checks of the expert-order row operators and the low-rank adapters:
every refusal comes before any launch (no GPU needed)."""
import ctypes

import pytest

import quantized_gemm_int4_amd as hm

P = ctypes.c_void_p
GOOD, ODD8, ODD2 = P(0x100000), P(0x100008), P(0x100002)     # never dereferenced: the calls return first
NULL, SHAPE, ALIGN, WORKSPACE, ABI = 1, 2, 3, 5, 7


def _call(fn, *args):
    return getattr(hm.lib, fn)(*args)


def _with(args, i, v):
    return args[:i] + [v] + args[i + 1:]


DISPATCH = [GOOD, GOOD, 4, 2, 8, 64, GOOD, GOOD, GOOD, GOOD, GOOD, None, 0, None]
GRAD_ROWS = [GOOD, GOOD, 4, 2, 64, GOOD, None]
COLLECT = [GOOD, GOOD, GOOD, 4, 2, 64, GOOD, None]
COLLECT_GRAD = [GOOD, GOOD, GOOD, GOOD, 4, 2, 64, GOOD, GOOD, None]


@pytest.mark.parametrize("fn,args,ptrs,t,topk,n", [
    ("hm_moe_dispatch", DISPATCH, (0, 1, 6, 7, 8, 9, 10), 2, 3, 5),
    ("hm_moe_dispatch_grad", GRAD_ROWS, (0, 1, 5), 2, 3, 4),
    ("hm_moe_collect", COLLECT, (0, 1, 2, 6), 3, 4, 5),
    ("hm_moe_collect_grad", COLLECT_GRAD, (0, 1, 2, 3, 7, 8), 4, 5, 6)])
def test_row_operator_refusals(fn, args, ptrs, t, topk, n):
    for i in ptrs:
        assert _call(fn, *_with(args, i, None)) == NULL, i
        assert _call(fn, *_with(args, i, ODD2)) == ALIGN, i
    assert _call(fn, *_with(args, t, -1)) == SHAPE
    assert _call(fn, *_with(args, topk, 0)) == SHAPE
    assert _call(fn, *_with(args, n, 0)) == SHAPE
    assert _call(fn, *_with(args, n, (1 << 24) + 1)) == SHAPE
    assert _call(fn, *_with(args, t, 1 << 24)) == SHAPE              # blocks of a launch
    assert _call(fn, *_with(_with(args, t, 1 << 23), topk, 512)) == SHAPE     # pairs beyond 2^31
    empty = args
    for i in ptrs:
        empty = _with(empty, i, None)
    assert _call(fn, *_with(empty, t, 0)) == 0                        # t = 0: a no-op, pointers not looked at


def test_dispatch_experts_and_workspace():
    assert _call("hm_moe_dispatch", *_with(DISPATCH, 4, 0)) == SHAPE
    assert _call("hm_moe_dispatch", *_with(DISPATCH, 4, 513)) == SHAPE
    assert _call("hm_moe_dispatch", *_with(DISPATCH, 4, 1)) == SHAPE      # topk above the experts
    need = hm.hm_moe_dispatch_workspace_size(100000, 2, 8)
    assert need > 0 and hm.hm_moe_dispatch_workspace_size(4, 2, 8) == 0
    big = _with(DISPATCH, 2, 100000)
    assert _call("hm_moe_dispatch", *big) == NULL
    assert _call("hm_moe_dispatch", *_with(_with(big, 11, GOOD), 12, need - 1)) == WORKSPACE
    assert _call("hm_moe_dispatch", *_with(_with(big, 11, ODD8), 12, need)) == ALIGN
    assert _call("hm_moe_dispatch_workspace_size", 4, 2, 8, None) == NULL
    for bad in ((-1, 2, 8), (4, 0, 8), (4, 9, 8), (4, 2, 513)):
        with pytest.raises(hm.HmError):
            hm.hm_moe_dispatch_workspace_size(*bad)


def _desc(**kw):
    d = hm.lora_desc(256, 512, 16, 4)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


BAD_DESC = [(dict(abi=1), ABI), (dict(rank=0), SHAPE), (dict(rank=12), SHAPE), (dict(rank=136), SHAPE),
            (dict(num_adapters=0), SHAPE), (dict(num_adapters=513), SHAPE), (dict(reserved=1), SHAPE),
            (dict(n=0), SHAPE), (dict(n=(1 << 24) + 1), SHAPE), (dict(k=0), SHAPE), (dict(k=200), SHAPE),
            (dict(k=(1 << 20) + 128), SHAPE)]


def _lora(d, m=4, x=GOOD, ids=GOOD, a=GOOD, b=GOOD, sc=GOOD, base=GOOD, y=GOOD, h=None, ws=GOOD, wsb=1 << 30):
    return _call("hm_lora", ctypes.byref(d) if d else None, x, ids, a, b, sc, m, base, y, h, ws, wsb, None)


def _grad(d, m=4, dy=GOOD, x=GOOD, h=GOOD, ids=GOOD, a=GOOD, b=GOOD, sc=GOOD, base=GOOD, dx=GOOD, da=GOOD, db=GOOD,
          ws=GOOD, wsb=1 << 30):
    return _call("hm_lora_grad", ctypes.byref(d) if d else None, dy, x, h, ids, a, b, sc, m, base, dx, da, db, ws, wsb,
                 None)


@pytest.mark.parametrize("kw,code", BAD_DESC)
def test_lora_descriptor_refusals(kw, code):
    d, sz = _desc(**kw), ctypes.c_size_t()
    assert _lora(d) == code and _grad(d) == code
    assert _call("hm_lora_workspace_size", ctypes.byref(d), 4, ctypes.byref(sz)) == code
    assert _call("hm_lora_grad_workspace_size", ctypes.byref(d), 4, ctypes.byref(sz)) == code


def test_lora_argument_refusals():
    d, sz = _desc(), ctypes.c_size_t()
    assert _lora(None) == NULL and _grad(None) == NULL
    for fn in ("hm_lora_workspace_size", "hm_lora_grad_workspace_size"):
        assert _call(fn, None, 4, ctypes.byref(sz)) == NULL
        assert _call(fn, ctypes.byref(d), 4, None) == NULL
        assert _call(fn, ctypes.byref(d), -1, ctypes.byref(sz)) == SHAPE
        assert _call(fn, ctypes.byref(d), (1 << 20) + 1, ctypes.byref(sz)) == SHAPE
        assert _call(fn, ctypes.byref(d), 0, ctypes.byref(sz)) == 0 and sz.value == 0
    for k in ("x", "ids", "a", "b", "sc", "y"):
        assert _lora(d, **{k: None}) == NULL, k
    for k in ("dy", "x", "h", "ids", "a", "b", "sc", "da", "db"):
        assert _grad(d, **{k: None}) == NULL, k
    for k in ("x", "a", "b", "base", "y", "h"):
        assert _lora(d, **{k: ODD8}) == ALIGN, k
    for k in ("dy", "x", "h", "a", "b", "base", "dx", "da", "db"):
        assert _grad(d, **{k: ODD8}) == ALIGN, k
    for k in ("ids", "sc"):
        assert _lora(d, **{k: ODD2}) == ALIGN and _grad(d, **{k: ODD2}) == ALIGN, k
    for m in (-1, (1 << 20) + 1):
        assert _lora(d, m=m) == SHAPE and _grad(d, m=m) == SHAPE
    assert _lora(d, m=0, x=None, ids=None, a=None, b=None, sc=None, y=None, ws=None) == 0
    assert _grad(d, m=0, da=None) == NULL                       # da and db are written even for no rows


@pytest.mark.parametrize("m", [1, 31, 33, 600, 5000])
def test_lora_workspace_checks(m):
    d = hm.lora_desc(1000, 512, 64, 40)
    need = hm.hm_lora_workspace_size(d, m)
    if need:
        assert _lora(d, m=m, ws=None) == NULL
        assert _lora(d, m=m, ws=ODD8) == ALIGN
        assert _lora(d, m=m, wsb=need - 1) == WORKSPACE
    need = hm.hm_lora_grad_workspace_size(d, m)
    assert _grad(d, m=m, ws=None) == NULL
    assert _grad(d, m=m, ws=ODD8) == ALIGN
    assert _grad(d, m=m, wsb=need - 1) == WORKSPACE


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        hm.hm_moe_dispatch(x, ids, 8)
    with pytest.raises(ValueError):
        hm.hm_moe_collect(x, torch.zeros(2, 2), ids)
    with pytest.raises(ValueError):
        hm.hm_lora(hm.lora_desc(8, 128, 8, 1), x, ids, x, x, x)
