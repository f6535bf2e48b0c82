"""Overlapping arrays of the low-rank adapters: an output over an array that
other blocks of the call still read is refused before any launch (no GPU
needed); the two in-place forms pass the checks."""
import ctypes

import pytest

import quantized_gemm_int4_amd as hm

pytestmark = pytest.mark.skipif(hm.torch.cuda.device_count() > 0, reason="the addresses are no arrays: nothing may run")
UNSUPPORTED = 4
M, N, K, RANK, L = 24, 256, 256, 16, 4
SIZES = dict(x=2 * M * K, ids=4 * M, a=2 * L * RANK * K, b=2 * L * N * RANK, sc=4 * L, base=2 * M * N, y=2 * M * N,
             h=4 * M * RANK, dy=2 * M * N, dxb=2 * M * K, dx=2 * M * K, da=2 * L * RANK * K, db=2 * L * N * RANK, ws=1 << 30)


def _place(**over):
    """Addresses (never dereferenced) 1 MiB or more apart, and those of `over`."""
    at, out = 1 << 40, {}
    for name, size in SIZES.items():
        out[name] = at
        at += (size + (1 << 20)) // (1 << 20) * (1 << 20)
    for name, (of, off) in over.items():
        out[name] = out[of] + off
    return {k: ctypes.c_void_p(v) for k, v in out.items()}


def _lora(m, **over):
    p = _place(**over)
    d = hm.lora_desc(N, K, RANK, L)
    return hm.lib.hm_lora(ctypes.byref(d), p["x"], p["ids"], p["a"], p["b"], p["sc"], m, p["base"], p["y"], p["h"], p["ws"],
                          SIZES["ws"], None)


def _grad(**over):
    p = _place(**over)
    d = hm.lora_desc(N, K, RANK, L)
    return hm.lib.hm_lora_grad(ctypes.byref(d), p["dy"], p["x"], p["h"], p["ids"], p["a"], p["b"], p["sc"], M, p["dxb"],
                               p["dx"], p["da"], p["db"], p["ws"], SIZES["ws"], None)


@pytest.mark.parametrize("m", [3, M])
@pytest.mark.parametrize("of", ["x", "a", "b", "base"])
def test_y_over_an_input_is_refused(m, of):
    for off in (0, 16, -16, SIZES[of] // M * m - 16 if of in ("x", "base") else SIZES[of] - 16, 16 - 2 * m * N):
        if of == "base" and off == 0:
            continue                                            # in place
        assert _lora(m, y=(of, off)) == UNSUPPORTED, off


@pytest.mark.parametrize("out", ["dx", "da", "db"])
@pytest.mark.parametrize("of", ["dy", "x", "h", "a", "b", "dxb"])
def test_gradient_over_an_input_is_refused(out, of):
    for off in (0, 16, -16, SIZES[of] - 16, 16 - SIZES[out]):
        if out == "dx" and of == "dxb" and off == 0:
            continue                                            # in place
        assert _grad(**{out: (of, off)}) == UNSUPPORTED, off


def test_neighbours_and_in_place_pass():
    ok = 6                                                      # past every check: the launch is what fails
    assert _lora(M) == ok and _lora(3) == ok and _grad() == ok
    assert _lora(M, y=("base", 0)) == ok and _grad(dx=("dxb", 0)) == ok
    assert _lora(M, y=("x", SIZES["x"])) == ok and _lora(M, y=("x", -SIZES["y"])) == ok
    assert _grad(dx=("dy", SIZES["dy"])) == ok and _grad(da=("h", -SIZES["da"])) == ok
