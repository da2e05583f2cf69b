"""The cubic that takes a share of the tcgen05 forward pass' exponentials, step by step in fp32 with the source's own
constants, against exp2."""
import os
import re

import numpy as np
import pytest

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bi_level_routing_b200", "csrc", "bra_diff.cuh")


def fma(a, b, c):  # the product of two fp32 values is exact in 64 bits
    return (a.astype(np.float64) * b.astype(np.float64) + c.astype(np.float64)).astype(np.float32)


@pytest.fixture(scope="module")
def poly():
    """poly_exp2 of an fp32 array, from the source: floor of x, shift, cubic from the highest coefficient down."""
    text = open(HEADER).read()
    body = text[text.index("poly_exp2(float2 x)"):]
    body = body[:body.index("\n}")]
    floor = np.float32(re.search(r"fmaxf\(x\.x, (-[0-9.]+)f\)", body)[1])
    coefficients = [np.float32(c) for c in re.findall(r"make_float2\((0\.\d{6,})f, \1f\)", body)]
    assert len(coefficients) == 4 and body.count("12582912.f") == 4

    def run(x):
        x = np.maximum(np.asarray(x, np.float32), floor)
        n = x + np.float32(12582912)
        f = (x - (n - np.float32(12582912))).astype(np.float32)
        p = np.full_like(x, coefficients[0])
        for c in coefficients[1:]:
            p = fma(p, f, np.full_like(x, c))
        return (p.view(np.uint32) + (n.view(np.uint32) << np.uint32(23))).view(np.float32)

    return run


def bf16(x):
    """fp32 rounded to bf16, to nearest even."""
    u = x.view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32)).view(np.float32)


def test_relative_error(poly):
    x = np.concatenate([np.linspace(-125.9, 8.5, 400001), np.linspace(-1, 1, 200001), np.arange(-125, 9)]).astype(np.float32)
    want = np.exp2(x.astype(np.float64))
    # the fit's 7.5e-5 and four fp32 roundings; a 26th of half a bf16 step
    assert np.abs(poly(x) / want - 1).max() <= 7.5e-5 + 4 * 2.0 ** -24


def test_least_values(poly):
    """Below -126 nothing is above 2^-126 or below 0, and what a mask leaves (-inf, the lowest values) is 0 in bf16."""
    x = np.linspace(-130, -125.9, 100001).astype(np.float32)
    y = poly(x)
    assert (y >= 0).all() and (y[x <= -126] <= np.float32(2.0 ** -126)).all()
    masked = np.array([-np.inf, np.finfo(np.float32).min, -1e9, -200.0, -127.0], np.float32)
    assert (bf16(poly(masked)) == 0).all()
