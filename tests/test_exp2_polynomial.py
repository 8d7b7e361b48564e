"""The exponentials that the cross attention kernel forms on the FMA pipe: its coefficients, read
from the source, evaluated step by step in fp32 as the kernel does (no GPU)."""

import os
import re

import numpy as np
import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantization_head_b200", "csrc",
                      "raw_cross.cu")
F = np.float32


def coefficients():
    """(fp16 weights', bf16 weights') coefficients, highest power first."""
    text = open(SOURCE).read()
    body = text[text.index("uint64_t exp2_pair(uint64_t x)"):]
    body = body[:body.index("return mul2")]
    first, second = body.split("} else {")
    number = r"pair\((-?[\d.]+)f, \1f\)"

    def of(part):
        lines = [s for s in part.splitlines() if "p = fma2" in s]
        return [F(c) for s in lines for c in re.findall(number, s)]

    return of(first), of(second)


def exp2(x, coef):
    # (fp64 holds the product of two fp32 numbers, so each step rounds once)
    x = np.maximum(x, F(-127.0))
    t = (x + F(12582912.0)).astype(F)
    n = (t - F(12582912.0)).astype(F)
    f = (x - n).astype(F)
    p = np.full_like(x, coef[0])
    for c in coef[1:]:
        p = (p.astype(np.float64) * f.astype(np.float64) + np.float64(c)).astype(F)
    scale = ((t.view(np.uint32) << np.uint32(23)) + np.uint32(0x3F800000)).view(F)
    return p * scale


@pytest.mark.parametrize("which,degree,bits", [(0, 4, 18.5), (1, 3, 13.7)])
def test_the_polynomials_are_as_exact_as_stated(which, degree, bits):
    coef = coefficients()[which]
    assert len(coef) == degree + 1
    f = np.linspace(-0.5, 0.5, 200001)
    p = np.polyval([np.float64(c) for c in coef], f)
    assert np.abs(p / np.exp2(f) - 1.0).max() <= 2.0 ** -bits
    # with the roundings of fp32: one for each fused step of a value near 1, halved or less by
    # the powers of f that follow, so less than two units in all
    x = np.concatenate([np.linspace(-126.0, 16.0, 1000003), np.arange(-126, 17), np.arange(-126, 16) + 0.5]).astype(F)
    err = np.abs(exp2(x, coef).astype(np.float64) / np.exp2(x.astype(np.float64)) - 1.0).max()
    assert err <= 2.0 ** -bits + 2.0 ** -23


def test_a_score_of_minus_infinity_weighs_nothing():
    for coef in coefficients():
        x = np.array([-np.inf, -1e30, -127.0, -126.75], F)
        assert not exp2(x, coef).any()
        assert (exp2(np.array([-126.0, -126.25], F), coef) > 0).all()
