"""Differential attention where most scores vanish: keys masked by scores of -inf, or so low that they count as
nothing, against the 64-bit definition over the keys that are left."""
import math

import pytest
import torch

import bi_level_routing_b200 as bra
import reference64 as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HEAD = 4.0  # the query's value in the channel (one a map) that sets all scores of a key


def masked_inputs(hr, wr, n_win, hd, dtype, dead_first, low, level, seed):
    """One image and head whose rows name every region in order. The keys of half the regions (of half the tokens
    of a single region), the first or the last, score -inf by `low` in one channel of each map; the others score
    about `level` in units of log2. Returns the call's inputs and which tokens' keys are masked."""
    g = torch.Generator().manual_seed(seed)
    H, W, R, d = hr * n_win, wr * n_win, n_win * n_win, hd // 2
    q, k, v, dout = (0.5 * torch.randn((1, H, W, hd), generator=g) for _ in range(4))
    tok = ref.region_tokens(H, W, n_win)
    if R > 1:
        half = tok[:(R + 1) // 2] if dead_first else tok[R // 2:]
        gone = torch.cat(half)
    else:
        gone = tok[0][:len(tok[0]) // 2] if dead_first else tok[0][len(tok[0]) // 2:]
    dead = torch.zeros(H * W, dtype=torch.bool)
    dead[gone] = True
    for c in (0, d):
        q[..., c] = HEAD
        k[..., c] = level * math.log(2) * math.sqrt(d) / HEAD
        k.view(-1, hd)[dead, c] = low
    q, k, v, dout = (t.to(dtype).cuda() for t in (q, k, v, dout))
    idx = torch.arange(R, dtype=torch.int32).expand(1, R, R).contiguous().cuda()
    return q, k, v, idx, torch.tensor([0.6], device="cuda"), dout, dead


def masked_reference(q, k, v, lam, dout, n_win, dead):
    """The definition over the keys that are not masked, whose probabilities are exactly 0, with reference64's bounds."""
    low = 2.0 ** -8 if q.dtype == BF16 else 0.0
    shape, hd = q.shape, q.shape[-1]
    d, l = hd // 2, float(lam[0])
    scale = 1 / math.sqrt(d)
    q, k, v, do = (t.cpu().double().view(-1, hd) for t in (q, k, v, dout))
    src = torch.cat(ref.region_tokens(shape[1], shape[2], n_win))
    src = src[~dead[src]]
    kk, vv, n, nq = k[src], v[src], len(src), len(q)
    halves = (slice(0, d), slice(d, hd))
    p = [torch.softmax(q[:, i] @ kk[:, i].T * scale, -1) for i in halves]
    mag = max(float((q[:, i].abs() @ kk[:, i].abs().T).max()) * scale for i in halves)
    c = 2 * (d + 6) * 2.0 ** -24 * mag + 2.0 ** -20 + 2 * (len(dead) + 8) * 2.0 ** -24
    both = p[0] + abs(l) * p[1]
    z = lambda: torch.zeros_like(q)
    res = {"out": (p[0] - l * p[1]) @ vv, "out_tol": (low + c) * (both @ vv.abs())}
    for name in ("dq", "dk", "dv"):
        res[name], res[name + "_tol"] = z(), z()
    res["dv"][src] = (p[0] - l * p[1]).T @ do
    res["dv_tol"][src] = (low + c + nq * 2.0 ** -24) * (both.T @ do.abs())
    dp, m = do @ vv.T, do.abs() @ vv.abs().T
    for i, w in ((0, 1.0), (1, -l)):
        D, Dm = (p[i] * dp).sum(-1, keepdim=True), (p[i] * m).sum(-1, keepdim=True)
        ds = p[i] * (dp - D)
        err = p[i] * (low * (dp - D).abs() + 2 * (c + (hd + 4) * 2.0 ** -24) * (m + Dm))
        s = halves[i]
        res["dq"][:, s] = w * scale * ds @ kk[:, s]
        res["dq_tol"][:, s] = abs(w) * scale * err @ kk[:, s].abs()
        res["dk"][src, s] = w * scale * ds.T @ q[:, s]
        res["dk_tol"][src, s] = abs(w) * scale * (err + nq * 2.0 ** -24 * ds.abs()).T @ q[:, s].abs()
    res["dlam"], res["dlam_tol"] = -D.sum().view(1), 2 * (c + (hd + 4) * 2.0 ** -24) * Dm.sum().view(1)
    return {name: t if name.startswith("dlam") else t.view(shape) for name, t in res.items()}


# hr, wr, n_win, hd, dtype: more keys than one tile in every kernel family, forward and backward
MASKED = [
    # CUDA cores: one-token regions, small ones, larger ones with few and many keys, wide heads
    (1, 1, 16, 32, F32), (3, 3, 4, 64, F32), (5, 5, 3, 48, F32), (5, 7, 3, 64, F32), (11, 12, 1, 128, F32),
    # one tile
    (1, 1, 7, 64, BF16), (2, 2, 3, 32, BF16),
    # mma.sync with one, two and four warps a region, and heads that only it takes
    (2, 2, 8, 64, BF16), (4, 5, 3, 32, BF16), (7, 7, 2, 64, BF16), (9, 9, 2, 24, BF16), (6, 6, 2, 128, BF16),
    # tcgen05, both head paddings; one region of two key tiles, of which one warpgroup of the backward pass meets
    # only masked keys; keys split over several CTAs
    (9, 9, 2, 64, BF16), (10, 10, 2, 128, BF16), (8, 16, 1, 64, BF16), (8, 16, 1, 128, BF16), (33, 32, 1, 64, BF16),
]


@pytest.mark.parametrize("dead_first", [True, False], ids=["masked_first", "masked_last"])
@pytest.mark.parametrize("low", ["-inf", "lowest"])
@pytest.mark.parametrize("shape", MASKED, ids=lambda s: "x".join(map(str, s)).replace("torch.", ""))
def test_scores_below_a_masked_tile(shape, low, dead_first):
    """A tile whose scores are all -inf says nothing about the maximum: the other keys' scores, some 150 binary
    orders below 0, make the row's softmax whether they come after it or before."""
    hr, wr, n_win, hd, dtype = shape
    low = float("-inf") if low == "-inf" else torch.finfo(dtype).min  # HEAD times the lowest value is -inf in fp32
    q, k, v, idx, lam, dout, dead = masked_inputs(hr, wr, n_win, hd, dtype, dead_first, low, -150.0, 5)
    want = masked_reference(q, k, v, lam, dout, n_win, dead)
    out = bra.diff_attend(q, k, v, idx, lam, 1, n_win)
    ref.check(out, want["out"], want["out_tol"], "out")
    got = dict(zip(("dq", "dk", "dv", "dlam"), bra.diff_attend_backward(q, k, v, idx, lam, dout, 1, n_win)))
    if math.isinf(low):  # dS k is 0 times -inf in the masks' channels
        rest = torch.ones(hd, dtype=torch.bool)
        rest[[0, hd // 2]] = False
        assert bool(torch.isnan(got["dq"][..., ~rest.cuda()]).all())
        got["dq"] = got["dq"][..., rest.cuda()]
        want["dq"], want["dq_tol"] = want["dq"][..., rest], want["dq_tol"][..., rest]
    for name, t in got.items():
        ref.check(t, want[name], want[name + "_tol"], name)
    assert bra.check_device_error() == 0


@pytest.mark.parametrize("dead_first", [True, False], ids=["masked_first", "masked_last"])
@pytest.mark.parametrize("shape", MASKED, ids=lambda s: "x".join(map(str, s)).replace("torch.", ""))
def test_values_of_masked_keys(shape, dead_first):
    """A key with a score of -inf has a probability of exactly 0: its value counts 0 times, the type's largest as well; an
    infinite one is 0 times infinity, NaN, in its own channel."""
    hr, wr, n_win, hd, dtype = shape
    q, k, v, idx, lam, dout, dead = masked_inputs(hr, wr, n_win, hd, dtype, dead_first, float("-inf"), 0.0, 6)
    v.view(-1, hd)[dead.cuda()] = torch.finfo(dtype).max
    want = masked_reference(q, k, v, lam, dout, n_win, dead)
    out = bra.diff_attend(q, k, v, idx, lam, 1, n_win)
    ref.check(out, want["out"], want["out_tol"], "out")
    v.view(-1, hd)[dead.cuda(), 5] = float("inf")
    out = bra.diff_attend(q, k, v, idx, lam, 1, n_win)
    assert bool(torch.isnan(out[..., 5]).all())
    rest = torch.arange(hd) != 5
    ref.check(out[..., rest.cuda()], want["out"][..., rest], want["out_tol"][..., rest], "out beside the infinity")
