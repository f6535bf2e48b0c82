"""Infinite and NaN inputs of the adapters against the definition, and values
that bf16 would round to infinity.

Each input array has one sign, so that no two infinities of a sum cancel and
every result of the definition is finite, an infinity or the NaN of an infinity
times a zero that the inputs hold.  Finite results are held to the bounds of
the parity tests: one rounding to bf16 (u = 2^-8 is half a step relative to the
value), and fp32 sums, off by 2^-24 of the sum of absolute terms per addition,
taken twice for the matrix unit's own rounding."""
import numpy as np
import pytest
import torch

from gpu_util import bf16_to_dev, bits_of, to_dev
from oracle import codecs, lora

pytestmark = pytest.mark.gpu
U = 2.0 ** -8

# m, n, k, rank, adapters: one-launch calls, calls without a grouping launch, units of 16, 32 and 64 rows
SHAPES = [(1, 40, 128, 8, 1), (5, 40, 256, 24, 2), (12, 70, 128, 64, 2), (12, 70, 128, 128, 2), (50, 40, 128, 16, 2),
          (50, 300, 256, 64, 3), (100, 40, 128, 16, 20), (150, 136, 256, 32, 6), (120, 72, 128, 128, 5),
          (300, 264, 256, 48, 2), (300, 72, 128, 128, 2), (700, 300, 256, 16, 1), (1400, 40, 128, 64, 1)]
PLACES = ["x", "dy", "h", "a", "b", "xn", "huge"]


def _val(bits):
    return codecs.bf16_value(bits).astype(np.float64)


def _bits(v):
    return codecs.bf16_rne_bits(np.float32(v).reshape(1))[0]


def _pos(r, *shape):
    """Positive bf16 values in [1/4, 1)."""
    return codecs.bf16_rne_bits(r.uniform(0.25, 0.999, shape).astype(np.float32))


def _case(m, n, k, rank, L, place):
    r = np.random.default_rng([m, n, k, rank, L])
    c = dict(x=_pos(r, m, k), a=_pos(r, L, rank, k), b=_pos(r, L, n, rank), base=_pos(r, m, n), dy=_pos(r, m, n),
             dxb=_pos(r, m, k), s=np.ones(L, np.float32), ids=r.integers(0, L, m).astype(np.int32),
             h=r.uniform(0.25, 1, (m, rank)).astype(np.float32))
    if m > 4:
        c["ids"][r.random(m) < 0.15] = -1
        c["ids"][1] = 0
    # every other row's h is a bf16 value, here and (one 1, a scale of 1) in the forward call
    c["h"][::2] = codecs.bf16_value(codecs.bf16_rne_bits(c["h"][::2]))
    c["x"][::2] = 0
    c["x"][::2, 5] = 0x3F80
    if m % 4 == 0:
        c["a"] ^= 0x8000                                        # h and the terms of dx negative
    if m % 3 == 0:
        c["b"] ^= 0x8000                                        # g too
    e = int(c["ids"][c["ids"] >= 0][0])
    mine = np.nonzero(c["ids"] == e)[0]
    inf = 0x7F80
    for row in {mine[0], mine[-1]}:                             # the first and last rows of its units
        if place == "x":
            c["x"][row, 5] = inf
        elif place == "dy":
            c["dy"][row, n // 2] = inf
        elif place == "h":
            c["h"][row, rank - 1] = np.inf
        elif place == "xn":
            c["x"][row, 7] = 0x7FC0
    if place == "a":
        c["a"][e, rank - 1, 5] = inf
    elif place == "b":
        c["b"][e, n - 1, rank // 2] = inf
    elif place == "huge":
        # h and g of 3.4e38, which bf16 would round to infinity, and products that bring them back into range
        c["s"][e] = np.float32(3.4e38)
        c["x"][mine], c["a"][e], c["b"][e] = 0, _bits(2.0 ** -12), _bits(2.0 ** -12)
        c["x"][mine, 3], c["a"][e, :, 3] = _bits(2.0 ** -20), _bits(2.0 ** 20)
        c["dy"][mine], c["dy"][mine, 0], c["b"][e, 0] = 0, _bits(2.0 ** -4), _bits(2.0 ** 4)
        c["h"][mine[0]] = np.float32(3.4e38)
    return c, e


def _same(got, ref, bound, terms, bf16=True):
    with np.errstate(all="ignore"):
        # an fp32 or bf16 result beyond the type's range is an infinity
        ref = np.where(np.abs(ref) > 3.4028235e38, np.sign(ref) * np.inf, ref)
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        inf = np.isinf(ref)
        assert np.array_equal(got[inf], ref[inf])
        ok = np.isfinite(ref)
        e = bound[ok] * terms * 2.0 ** -23
        assert (np.abs(got[ok] - ref[ok]) <= (U * (np.abs(ref[ok]) + e) if bf16 else 0) + e + 2.0 ** -120).all()


@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("m,n,k,rank,L", SHAPES)
def test_lora_infinities_as_in_the_definition(m, n, k, rank, L, place):
    import quantized_gemm_int4_amd as hm
    c, e = _case(m, n, k, rank, L, place)
    d = hm.lora_desc(n, k, rank, L)
    t = {key: bf16_to_dev(v) if v.dtype == np.uint16 else to_dev(v) for key, v in c.items()}
    h = torch.empty(m, rank, device="cuda")
    y = hm.hm_lora(d, t["x"], t["ids"], t["a"], t["b"], t["s"], base=t["base"], h=h)
    with np.errstate(all="ignore"):
        (ry, rh), (by, bh) = lora.lora_ref(_val(c["x"]), c["ids"], _val(c["a"]), _val(c["b"]), c["s"], _val(c["base"]))
    _same(h.cpu().numpy().astype(np.float64), rh, bh, k + 64, bf16=False)
    _same(_val(bits_of(y)), ry, by, k + 3 * rank + 64)
    got = hm.hm_lora_grad(d, t["dy"], t["x"], t["h"], t["ids"], t["a"], t["b"], t["s"], dx_base=t["dxb"])
    with np.errstate(all="ignore"):
        refs, bnds = lora.lora_grad_ref(_val(c["dy"]), _val(c["x"]), c["h"], c["ids"], _val(c["a"]), _val(c["b"]),
                                        c["s"], _val(c["dxb"]))
    for g, ref, bnd, terms in zip(got, refs, bnds, (n + 3 * rank + 64, n + 3 * m + 64, 3 * m + 64)):
        _same(_val(bits_of(g)), ref, bnd, terms)
