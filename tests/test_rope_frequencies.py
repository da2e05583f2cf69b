"""The frequency table's yarn scaling, pair by pair against the turns each makes over the trained positions."""
import math

import pytest
import torch

import bi_level_routing_b200 as bra


# n, base, trained_extent: every pair below one turn, both bounds inside the table, both past its end (raster numbers of
# large maps turn even the slowest pair several times), one below and one past
TABLES = [(8, 1e4, 4), (1, 1e4, 5), (8, 1e4, 7), (8, 1e4, 56), (8, 100.0, 56), (64, 1e4, 4096), (8, 1e4, 131072), (64, 1e4, 1 << 20),
          (32, 1e4, 65536), (16, 100.0, 16384), (1, 1e4, 300), (8, 1e4, 1 << 30), (64, 1e6, 1 << 30), (2, 1.5, 40)]


@pytest.mark.parametrize("factor", [1.0, 4.0, 32.0])
@pytest.mark.parametrize("n,base,extent", TABLES)
def test_yarn_every_pair(n, base, extent, factor):
    """More than 32 turns: kept. Less than one: divided by factor. Between: the ramp in the pair's number, from the last
    pair that is kept (or pair 0) to the first that is divided, wherever that would stand."""
    freqs, mscale = bra.rope_frequencies(n, base, "yarn", factor, extent)
    assert freqs.dtype == torch.float32 and freqs.shape == (n,)
    assert math.isclose(mscale, 0.1 * math.log(factor) + 1)
    number = lambda turns: n * math.log(extent / (turns * 2 * math.pi)) / math.log(base)  # the real pair number of so many turns
    low, high = max(math.floor(number(32)), 0), math.ceil(number(1))
    for i in range(n):
        full = base ** (-i / n)
        turns = extent * full / (2 * math.pi)
        part = 0.0 if turns > 32 else 1.0 if turns < 1 else (i - low) / (high - low) if high > low else 0.0
        want = full * (1 - part) + full / factor * part
        # the table is formed in 64 bits and rounded once
        assert math.isclose(float(freqs[i]), want, rel_tol=2.0 ** -24 + 1e-12), (i, turns, part)
