"""The bound that the two bf16 terms of dS keep in dq catches the mistakes it is there for: planted here in the 64-bit
form, on the CPU."""
import pytest
import torch

import dq_terms as dt
import reference64 as ref

SHAPES = [(4, 4, 1, 64), (1, 1, 8, 16), (5, 8, 1, 64), (8, 9, 1, 64), (8, 16, 1, 128), (4, 4, 2, 64), (16, 16, 1, 32), (6, 4, 4, 48)]


def two_terms(a, b):
    return [t + dt.rounded(x - t) for x, t in ((a, dt.truncated(a)), (b, dt.truncated(b)))]


MISTAKES = {
    "high term alone": lambda a, b: [dt.truncated(a), dt.truncated(b)],
    "one term, rounded": lambda a, b: [dt.rounded(a), dt.rounded(b)],
    "the other map's low term": lambda a, b: [dt.truncated(a) + dt.rounded(b - dt.truncated(b)), dt.truncated(b) + dt.rounded(a - dt.truncated(a))],
    "no low term in map 1": lambda a, b: [dt.truncated(a), two_terms(a, b)[1]],
    "no low term in map 2": lambda a, b: [two_terms(a, b)[0], dt.truncated(b)],
    "low term of every other key": lambda a, b: [t + dt.rounded(x - t) * (torch.arange(x.shape[-1]) % 2) for x, t in ((a, dt.truncated(a)), (b, dt.truncated(b)))],
}


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_bound_of_two_terms(shape):
    q, k, v, idx, lam, dout = dt.inputs(*shape)
    want = ref.diff(q, k, v, idx, lam, 1, shape[2], dout, low=2.0 ** -15)
    got = dt.dq_of(q, k, v, lam, dout, lambda a, b: (a, b))
    assert float((got - want["dq"]).abs().max()) < 1e-12
    ref.check(dt.dq_of(q, k, v, lam, dout, two_terms).to(torch.bfloat16), want["dq"], want["dq_tol"], "two terms")
    for name, split in MISTAKES.items():
        with pytest.raises(AssertionError, match="beyond its bound"):
            ref.check(dt.dq_of(q, k, v, lam, dout, split).to(torch.bfloat16), want["dq"], want["dq_tol"], name)
