"""The backward kernels where looser bounds would not tell: both bf16 terms of dS in dq, and the index sorted over
more than 256 regions in front of the tcgen05 kernels."""
import pytest
import torch

import bi_level_routing_b200 as bra
import dq_terms as dt
import reference64 as ref
from test_gpu_diff import BF16, check_all, make

pytestmark = pytest.mark.gpu

# hr, wr, n_win, hd. mma.sync: one tile of scores (one, two and four warps a region, half heads of up to 32), several
# tiles, wide heads, large regions of heads that only it takes; tcgen05: odd and even numbers of key tiles, both paddings
TERMS = [(1, 1, 8, 64), (4, 4, 1, 64), (4, 4, 2, 16), (3, 8, 1, 48), (5, 8, 1, 64), (4, 4, 4, 64), (4, 6, 2, 64), (6, 8, 2, 32), (4, 4, 2, 128),
         (4, 6, 2, 96), (8, 8, 2, 112), (10, 8, 2, 24), (8, 9, 1, 64), (8, 16, 1, 64), (10, 12, 2, 64), (8, 9, 1, 128), (8, 16, 1, 128),
         (10, 10, 2, 128), (16, 25, 1, 80), (16, 16, 1, 32)]


@pytest.mark.parametrize("shape", TERMS, ids=lambda s: "x".join(map(str, s)))
def test_dq_keeps_two_terms_of_ds(shape):
    """Within 2^-15 of each dS (dq_terms; the same bound refuses one term, or a low term in the wrong place)."""
    q, k, v, idx, lam, dout = dt.inputs(*shape)
    want = ref.diff(q, k, v, idx, lam, 1, shape[2], dout, low=2.0 ** -15)
    dq = bra.diff_attend_backward(*(t.cuda() for t in (q, k, v, idx, lam, dout)), 1, shape[2])[0]
    ref.check(dq, want["dq"], want["dq_tol"], "dq")


@pytest.mark.parametrize("shape", [(1, 9, 8, 17, 3, 1, 16), (1, 9, 8, 32, 2, 1, 16), (2, 8, 9, 17, 5, 1, 16)], ids=lambda s: "x".join(map(str, s)))
def test_sorted_index_of_many_regions(shape):
    """More regions than one pass of the sort's threads takes, with repeats, and a few that everything routes to."""
    q, k, v, idx, lam, dout = make(*shape, BF16, 80)
    idx[:, ::7, 0] = 3
    check_all(q, k, v, idx, lam, dout, shape[5], shape[3])
