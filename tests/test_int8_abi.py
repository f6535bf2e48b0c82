"""Argument checks of the 8-bit integer layers: every refusal comes before any
launch (no GPU needed)."""
import ctypes

import pytest

import quantized_gemm_int4_amd as hm

P = ctypes.c_void_p
NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5
STEP = 1 << 32                                                # addresses of arrays that do not meet; never dereferenced


def _p(i, off=0):
    return P(STEP * (i + 1) + off)


# name: (pointers in order, position of the sizes, positions of 4-byte aligned pointers, of outputs)
CALLS = {
    "hm_quant_int8_rows": (["x"], "mk", ["x8", "s"]),
    "hm_gemm_int8": (["x8", "xs", "w8", "ws_"], "mnk", ["y"]),
    "hm_gemm_int8_gated": (["x8", "xs", "w8", "ws_"], "mnk", ["h"]),
    "hm_gemm_int8_gated_grad": (["dh", "x8", "xs", "w8", "ws_"], "mnk", ["dgu"]),
    "hm_gemm_int8_grad": (["dy", "x8", "xs", "w8", "ws_"], "mnk", ["dx", "dw"]),
}
SMALL = {"xs", "ws_", "s"}                                     # fp32 scales: 4-byte aligned


def _call(fn, sizes=None, ws="big", wsb=1 << 40, **ptrs):
    ins, dims, outs = CALLS[fn]
    sizes = dict(dict(m=4, n=256, k=512), **(sizes or {}))
    at = {name: _p(i) for i, name in enumerate(ins + outs)}
    at.update(ptrs)
    args = [at[i] for i in ins] + [sizes[d] for d in dims] + [at[o] for o in outs]
    if fn != "hm_quant_int8_rows":
        args += [_p(20) if ws == "big" else ws, wsb]
    return getattr(hm.lib, fn)(*args, None)


@pytest.mark.parametrize("fn", CALLS)
def test_pointers(fn):
    ins, _, outs = CALLS[fn]
    for name in ins + outs:
        if not (fn == "hm_gemm_int8_grad" and name in outs):
            assert _call(fn, **{name: None}) == NULL, name
        i = (ins + outs).index(name)
        assert _call(fn, **{name: _p(i, 2 if name in SMALL else 8)}) == ALIGN, name
    for o in outs:                                             # an output over an input, at its start, middle and last bytes
        for name in ins:
            i = ins.index(name)
            if name not in SMALL:
                for off in (0, 16, 512):
                    assert _call(fn, **{o: _p(i, off)}) == UNSUPPORTED, (o, name, off)
    if len(outs) == 2:
        assert _call(fn, **{outs[1]: _p((ins + outs).index(outs[0]), 16)}) == UNSUPPORTED


@pytest.mark.parametrize("fn", [f for f in CALLS if f != "hm_quant_int8_rows"])
def test_sizes(fn):
    for bad in (dict(m=-1), dict(m=8388481), dict(n=0), dict(n=(1 << 22) + 2), dict(k=0), dict(k=200), dict(k=131072),
                dict(m=8388480, n=1 << 22)):
        assert _call(fn, bad) == SHAPE, bad
    sz = ctypes.c_size_t()
    size = getattr(hm.lib, fn + "_workspace_size")
    assert size(4, 256, 512, None) == NULL
    assert size(4, 256, 500, ctypes.byref(sz)) == SHAPE
    if "gated" in fn:
        assert _call(fn, dict(n=257)) == SHAPE and size(4, 257, 512, ctypes.byref(sz)) == SHAPE
    none = {p: None for p in sum(CALLS[fn][::2], [])}
    if fn == "hm_gemm_int8_grad":
        assert _call(fn, dict(m=0), dx=None, dw=None) == NULL
        none["dx"] = _p(1)                                     # only dw has something to write
    assert _call(fn, dict(m=0), ws=None, wsb=0, **none) == 0


def test_quant_sizes():
    assert _call("hm_quant_int8_rows", dict(m=-1)) == SHAPE
    assert _call("hm_quant_int8_rows", dict(k=0)) == SHAPE
    assert _call("hm_quant_int8_rows", dict(m=1 << 30, k=1 << 20)) == SHAPE
    assert _call("hm_quant_int8_rows", dict(m=0), x=None, x8=None, s=None) == 0


@pytest.mark.parametrize("fn", [f for f in CALLS if f != "hm_quant_int8_rows"])
@pytest.mark.parametrize("m", [1, 16, 17, 100, 700, 5000])
def test_workspace(fn, m):
    need = getattr(hm, fn + "_workspace_size")(m, 514, 1024)
    if need:
        s = dict(m=m, n=514, k=1024)
        assert _call(fn, s, ws=None) == NULL
        assert _call(fn, s, wsb=need - 1) == WORKSPACE
        assert _call(fn, s, ws=_p(20, 16)) == ALIGN
        assert _call(fn, s, ws=_p(0)) == UNSUPPORTED
    assert getattr(hm, fn + "_workspace_size")(0, 514, 1024) == 0


def test_gradient_of_one_side():
    fn, odd = "hm_gemm_int8_grad", dict(n=257)                 # (rows that are padded: a workspace is needed)
    assert hm.hm_gemm_int8_grad_workspace_size(4, 257, 512) > 0
    assert _call(fn, odd, dx=None, w8=None, ws_=None, wsb=0) == WORKSPACE      # the checks of the pointers are behind it
    assert _call(fn, odd, dw=None, x8=None, xs=None, wsb=0) == WORKSPACE
    assert _call(fn, odd, dx=None, dw=None) == NULL
    assert _call(fn, odd, dw=None, w8=None) == NULL and _call(fn, odd, dx=None, xs=None) == NULL


def test_plan():
    buf = ctypes.create_string_buffer(200)
    plan = hm.lib.hm_gemm_int8_plan
    for op in range(4):
        assert plan(op, 2000, 256, 512, buf, 200) == 0 and b"tiles" in buf.value
        assert plan(op, 0, 256, 512, buf, 200) == 0
        assert plan(op, 100, 256, 500, buf, 200) == SHAPE and plan(op, -1, 256, 512, buf, 200) == SHAPE
        assert plan(op, 100, 256, 512, None, 200) == NULL and plan(op, 100, 256, 512, buf, 0) == NULL
        assert plan(op, 100, 256, 512, buf, 4) == 0 and len(buf.value) < 4         # cut to the buffer
    assert plan(4, 100, 256, 512, buf, 200) == UNSUPPORTED and plan(-1, 100, 256, 512, buf, 200) == UNSUPPORTED
    assert "few" in hm.hm_gemm_int8_plan(hm.HM_INT8_GEMM, 1, 14336, 4096)
    for op in (hm.HM_INT8_GATED, hm.HM_INT8_GATED_GRAD):
        with pytest.raises(hm.HmError):
            hm.hm_gemm_int8_plan(op, 100, 257, 512)


def test_binding_refusals():
    import torch
    x8, s = torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError):
        hm.hm_gemm_int8(x8, s, x8, s)
    with pytest.raises(ValueError):
        hm.hm_quant_int8_rows(torch.zeros(4, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        hm.hm_gemm_int8_gated(x8, s, x8, s)
    with pytest.raises(ValueError):
        hm.hm_gemm_int8_gated_grad(x8, x8, s, x8, s)
    with pytest.raises(ValueError):
        hm.hm_gemm_int8_grad(x8, x8, s, x8, s)
