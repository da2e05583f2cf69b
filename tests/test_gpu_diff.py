"""Differential attention on the GPU against its 64-bit definition: every element of the output and of the
gradients within bounds that count the kernels' roundings (reference64), at the sizes and index rows where
it can go wrong."""
import math

import pytest
import torch

import bi_level_routing_b200 as bra
import reference64 as ref

pytestmark = pytest.mark.gpu


def make(B, hr, wr, n_win, topk, heads, hd, dtype, seed=0, spread=1.0, distinct=False):
    g = torch.Generator().manual_seed(seed)
    H, W, C, R = hr * n_win, wr * n_win, heads * hd, n_win * n_win
    q, k, v, dout = (torch.randn((B, H, W, C), generator=g) for _ in range(4))
    q, k = q * spread, k * spread
    if distinct:
        idx = torch.rand((B, R, R), generator=g).argsort(-1)[:, :, :topk].to(torch.int32)
    else:
        idx = torch.randint(0, R, (B, R, topk), generator=g, dtype=torch.int32)
    lam = torch.rand(heads, generator=g) * 1.2 - 0.2
    q, k, v, dout = (t.to(dtype).cuda() for t in (q, k, v, dout))
    return q, k, v, idx.contiguous().cuda(), lam.cuda(), dout


def check_all(q, k, v, idx, lam, dout, heads, n_win, what=""):
    want = ref.diff(q, k, v, idx, lam, heads, n_win, dout)
    out = bra.diff_attend(q, k, v, idx, lam, heads, n_win)
    ref.check(out, want["out"], want["out_tol"], f"{what} out")
    for name, t in zip(("dq", "dk", "dv", "dlam"), bra.diff_attend_backward(q, k, v, idx, lam, dout, heads, n_win)):
        ref.check(t, want[name], want[name + "_tol"], f"{what} {name}")
    assert bra.check_device_error() != 5, "a wait gave up"
    return want


BF16, F32 = torch.bfloat16, torch.float32
# B, hr, wr, n_win, topk, heads, hd: one token in all; one-token regions; regions below, at and past the kernels'
# tiles of 16, 32 and 64 rows, odd windows; one region of many tokens; every padding of a half head
SHAPES = [
    (1, 1, 1, 1, 1, 1, 32), (3, 1, 1, 1, 1, 2, 16), (2, 1, 1, 7, 49, 2, 64), (1, 1, 1, 5, 3, 3, 32), (2, 1, 1, 7, 5, 1, 64),
    (2, 2, 2, 7, 16, 2, 64), (1, 5, 3, 3, 2, 2, 48), (2, 4, 4, 7, 4, 2, 64), (1, 17, 1, 2, 3, 1, 64), (1, 4, 5, 3, 5, 2, 32),
    (2, 8, 4, 2, 2, 1, 128), (1, 3, 11, 2, 4, 2, 64), (2, 8, 8, 3, 1, 1, 64), (1, 9, 7, 2, 3, 2, 80), (1, 10, 10, 2, 2, 1, 96),
    (1, 13, 10, 1, 1, 2, 64), (1, 1, 257, 1, 1, 1, 64), (1, 16, 17, 1, 1, 1, 128), (1, 8, 8, 2, 4, 1, 112), (1, 6, 6, 2, 3, 2, 16),
    # small maps in batches large enough for the dense mode
    (37, 1, 1, 7, 9, 1, 64), (30, 2, 2, 4, 5, 4, 16), (60, 2, 4, 2, 3, 8, 16), (200, 1, 1, 3, 9, 1, 128), (23, 8, 1, 2, 4, 20, 48),
    (1, 16, 16, 1, 1, 1, 32), (1, 12, 11, 2, 3, 2, 64), (2, 16, 8, 2, 4, 1, 128), (1, 15, 9, 3, 5, 1, 64), (1, 1, 128, 1, 1, 2, 128),
    (1, 20, 13, 2, 3, 1, 128), (1, 8, 8, 3, 5, 2, 64), (1, 9, 9, 2, 2, 2, 16), (1, 11, 12, 2, 3, 1, 48), (1, 10, 7, 3, 4, 1, 112), (2, 8, 9, 2, 4, 1, 32), (1, 129, 1, 2, 2, 2, 64), (1, 1, 3, 16, 7, 1, 32), (2, 1, 2, 32, 5, 1, 16),
]
ODD_HEADS = [(1, 3, 3, 2, 3, 2, 8), (1, 5, 2, 2, 2, 1, 24), (1, 1, 1, 3, 9, 2, 40), (1, 9, 8, 1, 1, 1, 56), (1, 4, 4, 2, 2, 1, 120)]


@pytest.mark.parametrize("shape", SHAPES + ODD_HEADS, ids=lambda s: "x".join(map(str, s)))
def test_bf16(shape):
    B, hr, wr, n_win, topk, heads, hd = shape
    check_all(*make(*shape, BF16), heads, n_win)


@pytest.mark.parametrize("shape", SHAPES[::2] + ODD_HEADS, ids=lambda s: "x".join(map(str, s)))
def test_f32(shape):
    B, hr, wr, n_win, topk, heads, hd = shape
    check_all(*make(*shape, F32), heads, n_win)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rs", [(1, 1), (3, 4), (4, 6), (9, 9), (12, 12)])
def test_bad_entries_and_empty_rows(dtype, rs):
    """Entries outside [0, R) contribute nothing and are flagged; a row with none left gives 0 and takes part
    in no gradient; a region that nothing routes to has gradients 0."""
    heads, n_win, topk, hd = 2, 3, 4, 64
    q, k, v, idx, lam, dout = make(100 if rs == (1, 1) else 2, *rs, n_win, topk, heads, hd, dtype, 3)  # 100: the dense mode
    idx[idx == 5] = 4  # nothing routes to region 5
    idx[0, 2] = torch.tensor([-1, 9, 1 << 30, -(1 << 31)], dtype=torch.int32)
    idx[1, 7, 0], idx[1, 7, 3], idx[0, 0, 1] = -7, 9, 100
    bra.check_device_error()
    bra.diff_attend(q, k, v, idx, lam, heads, n_win)
    assert bra.check_device_error() == 4
    want = check_all(q, k, v, idx, lam, dout, heads, n_win, "bad entries")
    bra.diff_attend_backward(q, k, v, idx, lam, dout, heads, n_win)
    assert bra.check_device_error() == 4
    tok = ref.region_tokens(q.shape[1], q.shape[2], n_win)
    out = bra.diff_attend(q, k, v, idx, lam, heads, n_win).flatten(1, 2)
    dq, dk, dv, _ = (t.flatten(1, 2) if t.dim() == 4 else t for t in
                     bra.diff_attend_backward(q, k, v, idx, lam, dout, heads, n_win))
    assert bool((out[0, tok[2]] == 0).all()) and bool((dq[0, tok[2]] == 0).all())
    assert bool((dk[:, tok[5]] == 0).all()) and bool((dv[:, tok[5]] == 0).all())
    assert float(want["out"].abs().max()) > 0
    assert bra.check_device_error() == 4
    # every entry of the batch bad
    idx.fill_(-1)
    out = bra.diff_attend(q, k, v, idx, lam, heads, n_win)
    grads = bra.diff_attend_backward(q, k, v, idx, lam, dout, heads, n_win)
    assert bool((out == 0).all()) and all(bool((t == 0).all()) for t in grads)
    assert bra.check_device_error() == 4


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rs", [(1, 1), (3, 5), (5, 9), (8, 9), (11, 13)])
def test_not_finite_outside_the_routed_regions(dtype, rs):
    """NaN and infinities in a region that nobody routes to change nothing elsewhere."""
    heads, n_win, hd = 1, 3, 64
    q, k, v, idx, lam, dout = make(200 if rs == (1, 1) else 1, *rs, n_win, 2, heads, hd, dtype, 4)  # 200: the dense mode
    idx[idx == 4] = 3
    want = ref.diff(q, k, v, idx, lam, heads, n_win, dout)
    tok = ref.region_tokens(q.shape[1], q.shape[2], n_win)
    for bad in (float("nan"), float("inf"), torch.finfo(dtype).min):
        k2, v2 = k.clone(), v.clone()
        k2.view(len(q), -1, hd)[:, tok[4]] = bad
        v2.view(len(q), -1, hd)[:, tok[4]] = bad
        out = bra.diff_attend(q, k2, v2, idx, lam, heads, n_win)
        ref.check(out, want["out"], want["out_tol"], f"{bad} out")
        for name, t in zip(("dq", "dk", "dv", "dlam"),
                           bra.diff_attend_backward(q, k2, v2, idx, lam, dout, heads, n_win)):
            ref.check(t, want[name], want[name + "_tol"], f"{bad} {name}")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 7, 5, 1, 64), (37, 1, 1, 7, 5, 1, 64), (1, 4, 4, 3, 2, 1, 64), (1, 3, 4, 3, 7, 1, 32), (1, 9, 9, 2, 2, 1, 64), (1, 16, 15, 1, 1, 1, 128)],
                         ids=lambda s: "x".join(map(str, s)))
def test_not_finite_scores_make_their_rows_nan(shape, dtype):
    """A NaN or infinite element of a query or a key: outputs and gradients are not finite exactly where the 64-bit
    definition's are (a query's own row; every query that names the key's region), and elsewhere what they were."""
    B, hr, wr, n_win, topk, heads, hd = shape
    for where, bad in (("q", "nan"), ("k", "nan"), ("k", "inf"), ("q", "-inf")):
        q, k, v, idx, lam, dout = make(*shape, dtype, 50)
        idx[0, 0] = n_win * n_win - 1
        t = {"q": q, "k": k}[where]
        t.view(-1, hd)[-1 if where == "k" else 0, 3] = float(bad)
        want = ref.diff(q, k, v, idx, lam, heads, n_win, dout)
        out = bra.diff_attend(q, k, v, idx, lam, heads, n_win)
        dq, dk, dv, _ = bra.diff_attend_backward(q, k, v, idx, lam, dout, heads, n_win)
        for name, got in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
            finite = torch.isfinite(want[name])
            assert 0 < int((~finite).sum()), (where, bad, name)
            assert torch.equal(torch.isfinite(got.cpu()), finite), (where, bad, name, int((torch.isfinite(got.cpu()) != finite).sum()))
            ok = finite & torch.isfinite(want[name + "_tol"])
            if bool(ok.any()):
                ref.check(got.cpu()[ok], want[name][ok], want[name + "_tol"][ok], f"{where} {bad} {name}")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_not_finite_values_reach_their_own_queries(dtype):
    """One infinite value: the queries whose rows name its region get an infinity or NaN in that channel,
    all others and all other channels what they had."""
    for hr, wr, n_win, hd in ((1, 1, 7, 64), (2, 3, 3, 32), (4, 4, 3, 64), (9, 9, 2, 64)):
        q, k, v, idx, lam, _ = make(40 if hr == 1 else 2, hr, wr, n_win, 2, 1, hd, dtype, 40)  # 40: the dense mode
        idx[1, 0] = 1  # one row that does not name region 0 and one that does
        idx[1, 1, 0] = 0
        before = bra.diff_attend(q, k, v, idx, lam, 1, n_win)
        v[1, 0, 0, 5] = float("inf")  # a token of region 0
        out = bra.diff_attend(q, k, v, idx, lam, 1, n_win)
        tok = ref.region_tokens(q.shape[1], q.shape[2], n_win)
        named = torch.zeros(q.shape[1] * q.shape[2], dtype=torch.bool)
        for r, t in enumerate(tok):
            named[t] = bool((idx[1, r] == 0).any())
        hit = torch.zeros(q.shape, dtype=torch.bool)
        hit[1, :, :, 5] = named.view(q.shape[1], q.shape[2])
        assert 0 < int(named.sum()) < named.numel()
        assert not bool(torch.isfinite(out.cpu()[hit]).any())
        assert torch.equal(out.cpu()[~hit], before.cpu()[~hit])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("spread", [0.0, 6.0, 1e-3])
def test_flat_and_peaked_maps(dtype, spread):
    """All scores equal (spread 0), and scores some hundreds apart."""
    for shape in ((1, 3, 3, 3, 5, 2, 64), (1, 12, 13, 1, 1, 1, 64), (1, 12, 13, 1, 1, 1, 128)):
        check_all(*make(*shape, dtype, 9, spread), shape[5], shape[3], f"spread {spread}")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_special_weights(dtype):
    """lam = 0 leaves the first map, lam = 1 with equal halves cancels it."""
    q, k, v, idx, lam, dout = make(1, 5, 5, 2, 3, 2, 64, dtype, 5)
    lam.zero_()
    check_all(q, k, v, idx, lam, dout, 2, 2, "lam 0")
    lam.fill_(1.0)
    half = lambda t: t.unflatten(-1, (2, 2, 32))[..., :1, :].expand(*t.shape[:-1], 2, 2, 32).reshape(t.shape).contiguous()
    q, k = half(q), half(k)
    want = check_all(q, k, v, idx, lam, dout, 2, 2, "equal halves")
    assert float(want["out"].abs().max()) < 1e-12
    lam.copy_(torch.tensor([-2.5, 40.0]))
    check_all(q, k, v, idx, lam, dout, 2, 2, "large weights")


def test_many_slots_and_repeats():
    """Rows that name every region, some more than once, and one region in every slot: the same
    region's tokens count as often as they are named."""
    for dtype in (BF16, F32):
        q, k, v, idx, lam, dout = make(2, 2, 1, 8, 64, 1, 32, dtype, 6)
        idx[1, 3:9] = 11
        check_all(q, k, v, idx, lam, dout, 1, 8, "repeats")


def test_forward_diff_routes_like_route():
    for B, hr, wr, n_win, topk, heads, hd, dtype in ((2, 4, 4, 7, 4, 2, 64, BF16), (1, 1, 1, 7, 9, 2, 64, BF16),
                                                     (2, 3, 5, 4, 2, 1, 64, F32), (2, 8, 6, 1, 1, 1, 64, BF16)):
        q, k, v, _, lam, _ = make(B, hr, wr, n_win, topk, heads, hd, dtype, 7)
        out, idx = bra.forward_diff(q, k, v, lam, n_win, topk, heads)
        assert torch.equal(idx, bra.route(q, k, n_win, topk))
        assert torch.equal(out, bra.diff_attend(q, k, v, idx, lam, heads, n_win))
        want = ref.diff(q, k, v, idx, lam, heads, n_win)
        ref.check(out, want["out"], want["out_tol"], "forward_diff")
    # a row segment wider than the routing kernels take: one region needs no routing
    q, k, v, _, lam, _ = make(1, 2, 300, 1, 1, 1, 64, BF16, 8)
    out, idx = bra.forward_diff(q, k, v, lam, 1, 1, 1)
    assert int(idx.abs().max()) == 0
    want = ref.diff(q, k, v, idx, lam, 1, 1)
    ref.check(out, want["out"], want["out_tol"], "one wide region")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_same_bits_and_untouched_neighbours(dtype):
    """Two runs give the same bits; outputs are written in full and nothing past them is."""
    q, k, v, idx, lam, dout = make(3, 4, 4, 7, 4, 2, 64, dtype, 10, distinct=True)
    first = (bra.diff_attend(q, k, v, idx, lam, 2, 7),) + bra.diff_attend_backward(q, k, v, idx, lam, dout, 2, 7)
    guard = torch.full((q.numel() + 4096,), 7.0, dtype=dtype, device="cuda")
    bufs = [guard.clone() for _ in range(4)]
    view = lambda t: t[:q.numel()].view(q.shape)
    dlam = torch.full((2,), 7.0, device="cuda")
    bra.diff_attend(q, k, v, idx, lam, 2, 7, out=view(bufs[0]))
    bra.diff_attend_backward(q, k, v, idx, lam, dout, 2, 7, *map(view, bufs[1:]), dlam)
    for a, b in zip(first, [*map(view, bufs), dlam]):
        assert torch.equal(a, b)
    assert all(bool((t[q.numel():] == 7).all()) for t in bufs)


def test_streams_and_graphs():
    """On another stream, and captured: two graphs hold scratch of their own and replay with new inputs."""
    sets = [make(2, 4, 4, 3, 2, 2, 64, BF16, s) for s in (20, 21)]
    want = [(bra.diff_attend(q, k, v, i, l, 2, 3),) + bra.diff_attend_backward(q, k, v, i, l, do, 2, 3)
            for q, k, v, i, l, do in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q, k, v, i, l, do = sets[0]
        got = (bra.diff_attend(q, k, v, i, l, 2, 3),) + bra.diff_attend_backward(q, k, v, i, l, do, 2, 3)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    held = [[t.clone() for t in s] for s in sets]
    graphs, outs = [], []
    for q, k, v, i, l, do in held:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((bra.diff_attend(q, k, v, i, l, 2, 3),) + bra.diff_attend_backward(q, k, v, i, l, do, 2, 3))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))
    for dst, src in zip(held[0], sets[1]):
        dst.copy_(src)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], want[1]))


def test_refusals_in_python():
    q, k, v, idx, lam, dout = make(1, 4, 4, 2, 2, 2, 64, BF16)
    calls = [
        lambda: bra.diff_attend(q.transpose(1, 2), k, v, idx, lam, 2, 2),
        lambda: bra.diff_attend(q, k.float(), v, idx, lam, 2, 2),
        lambda: bra.diff_attend(q, k, v[:, :4], idx, lam, 2, 2),
        lambda: bra.diff_attend(q, k, v, idx.long(), lam, 2, 2),
        lambda: bra.diff_attend(q, k, v, idx[:, :3].contiguous(), lam, 2, 2),
        lambda: bra.diff_attend(q, k, v, idx, lam[:1], 2, 2),
        lambda: bra.diff_attend(q, k, v, idx, lam.cpu(), 2, 2),
        lambda: bra.diff_attend(q, k, v, idx, lam.double(), 2, 2),
        lambda: bra.diff_attend(q.half(), k.half(), v.half(), idx, lam, 2, 2),
        lambda: bra.diff_attend_backward(q, k, v, idx, lam, dout.float(), 2, 2),
        lambda: bra.diff_attend_backward(q, k, v, idx, lam, dout, 2, 2, dq=torch.empty_like(q, dtype=F32)),
        lambda: bra.forward_diff(q, k, v, lam, 2, 3, 2, idx=idx),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(bra.BraError):
        bra.diff_attend(q, k, v, idx, torch.ones(32, device="cuda"), 32, 2)  # heads of 4 channels
    with pytest.raises(bra.BraError):
        bra.forward_diff(q, k, v, lam, 2, 5, 2)  # topk > R


def test_long_map_sampled():
    """One region of 6000 tokens, 128-channel heads: sampled queries against the definition (each query's
    attention is over all keys), dlam and the keys' gradients through a random weighting of few queries."""
    H, W, heads, hd = 75, 80, 1, 128
    q, k, v, idx, lam, _ = make(1, H, W, 1, 1, heads, hd, BF16, 30)
    out = bra.diff_attend(q, k, v, idx, lam, heads, 1).view(-1, hd)
    pick = torch.tensor([0, 1, 63, 64, 127, 2999, 5950, 5999])
    dout = torch.zeros_like(q)
    g = torch.randn((len(pick), hd), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    dout.view(-1, hd)[pick] = g
    dq, dk, dv, dlam = bra.diff_attend_backward(q, k, v, idx, lam, dout, heads, 1)
    x, kk, vv = (t.view(-1, hd).cpu().double() for t in (q, k, v))
    gg, d, l = g.cpu().double(), hd // 2, float(lam[0])
    p = [torch.softmax(x[pick][:, s] @ kk[:, s].T / math.sqrt(d), -1) for s in (slice(0, d), slice(d, hd))]
    n = H * W
    mag = max(float((x[pick][:, s].abs() @ kk[:, s].abs().T).max()) / math.sqrt(d) for s in (slice(0, d), slice(d, hd)))
    c = 2 * (d + 6) * 2.0 ** -24 * mag + 2.0 ** -20 + 2 * (n + 8) * 2.0 ** -24
    both = p[0] + abs(l) * p[1]
    ref.check(out[pick], (p[0] - l * p[1]) @ vv, (2.0 ** -8 + c) * (both @ vv.abs()), "long out")
    ref.check(dv.view(-1, hd), (p[0] - l * p[1]).T @ gg, (2.0 ** -8 + c) * (both.T @ gg.abs()), "long dv")
    dp, m = gg @ vv.T, gg.abs() @ vv.abs().T
    for i, w, s in ((0, 1.0, slice(0, d)), (1, -l, slice(d, hd))):
        D, Dm = (p[i] * dp).sum(-1, keepdim=True), (p[i] * m).sum(-1, keepdim=True)
        ds, err = p[i] * (dp - D), p[i] * (2.0 ** -8 * (dp - D).abs() + 2 * (c + (hd + 4) * 2.0 ** -24) * (m + Dm))
        sc = w / math.sqrt(d)
        ref.check(dq.view(-1, hd)[pick][:, s], sc * ds @ kk[:, s], abs(sc) * err @ kk[:, s].abs(), f"long dq {i}")
        ref.check(dk.view(-1, hd)[:, s], sc * ds.T @ x[pick][:, s], abs(sc) * err.T @ x[pick][:, s].abs(), f"long dk {i}")
    ref.check(dlam, -D.sum().view(1), 2 * (c + (hd + 4) * 2.0 ** -24) * Dm.sum().view(1), "long dlam")
    zero = torch.ones(n, dtype=torch.bool)
    zero[pick] = False
    assert bool((dq.view(-1, hd)[zero.cuda()] == 0).all())


# One image, few query tiles and many keys: the keys of a tile are split over several CTAs and joined.
@pytest.mark.parametrize("shape", [(1, 33, 32, 1, 1, 1, 64), (1, 12, 11, 3, 9, 2, 32), (1, 47, 45, 1, 1, 1, 128), (1, 1, 2500, 1, 1, 1, 48),
                                   (1, 17, 16, 2, 4, 1, 80), (2, 70, 1, 4, 16, 1, 16)], ids=lambda s: "x".join(map(str, s)))
def test_split_keys(shape):
    B, hr, wr, n_win, topk, heads, hd = shape
    check_all(*make(*shape, BF16, 70), heads, n_win)


def test_split_keys_empty_and_infinite():
    """Splits without keys, rows without keys, splits whose scores are all -inf, rows of nothing else, and a NaN
    score among them. 9 regions of 132 tokens, 1188 keys in splits of at most 608."""
    hr, wr, n_win, topk, hd = 12, 11, 3, 9, 64
    q, k, v, idx, lam, _ = make(1, hr, wr, n_win, topk, 1, hd, BF16, 71)
    tok = ref.region_tokens(q.shape[1], q.shape[2], n_win)
    idx[:] = torch.arange(9, dtype=torch.int32, device="cuda")
    idx[0, 1, 2:] = -1                    # two regions' keys: the first split's
    idx[0, 2] = 9                         # none
    idx[0, 3, :7], idx[0, 3, 7:] = 99, 8  # the last region twice
    idx[0, 4] = 4                         # one region, nine times
    q[..., 0], k.view(-1, hd)[torch.cat(list(tok[:6])), 0] = 1.0, float("-inf")  # map 1 meets regions 6 to 8 only
    k.view(-1, hd)[tok[7][5], 40] = float("-inf")
    q[..., 40] = 0.5
    q.view(-1, hd)[tok[5][3], 40] = float("nan")
    out = bra.diff_attend(q, k, v, idx, lam, 1, n_win)
    assert bra.check_device_error() == 4  # the bad entries
    Q, K, V, l = (t.double().cpu().reshape(-1, hd) for t in (q, k, v, lam[:, None].expand(1, hd)))
    got = out.double().cpu().reshape(-1, hd)
    for r in range(9):
        named = [int(i) for i in idx[0, r] if 0 <= int(i) < 9]
        if not named:
            assert not bool(got[tok[r]].any())
            continue
        src = torch.cat([tok[i] for i in named])
        p1, p2 = (torch.softmax(Q[tok[r]][:, c] @ K[src][:, c].T / 32 ** 0.5, -1) for c in (slice(0, 32), slice(32, 64)))
        want = (p1 - l[0, 0] * p2) @ V[src]
        # P and the output are rounded to bf16 (2^-8 relative each); fp32 sums of 1188 terms
        tol = 2.0 ** -8 * ((p1 + l[0, 0].abs() * p2) @ V[src].abs() + want.abs()) + 1e-4
        fine = torch.isfinite(want)
        assert torch.equal(torch.isfinite(got[tok[r]]), fine), r
        assert bool(((got[tok[r]] - want).abs()[fine] <= tol[fine]).all()), r
        if r in (1, 4):  # map 1 has nothing but -inf
            assert not bool(fine.any())


def test_split_keys_captured_and_repeated():
    """The same bits on every run, in graphs with scratch of their own, and beside a whole batch in one piece."""
    q, k, v, idx, lam, _ = make(1, 40, 40, 1, 1, 1, 64, BF16, 72)
    first = bra.diff_attend(q, k, v, idx, lam, 1, 1)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(bra.diff_attend(q, k, v, idx, lam, 1, 1))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, bra.diff_attend(q, k, v, idx, lam, 1, 1))
    assert all(torch.equal(first, o) for o in outs)
    # 24 such images leave nothing to split: each element within the roundings of P and of the output, twice
    many = bra.diff_attend(*(t.expand(24, *t.shape[1:]).contiguous() for t in (q, k, v, idx)), lam, 1, 1)
    assert torch.equal(many[0], many[23])
    p = [torch.softmax(q.double().view(-1, 64)[:, c] @ k.double().view(-1, 64)[:, c].T / 32 ** 0.5, -1) for c in (slice(0, 32), slice(32, 64))]
    weight = (p[0] + lam.double().abs() * p[1]) @ v.double().view(-1, 64).abs()
    tol = 2 * 2.0 ** -8 * (weight + first.double().view(-1, 64).abs()) + 1e-4
    assert bool(((many[0] - first[0]).double().abs().view(-1, 64) <= tol).all())
    assert bra.kernels_per_call("bra_diff_attend", 1, 40, 40, 64, 1, 1, 1, BF16) == 2
    assert bra.kernels_per_call("bra_diff_attend", 24, 40, 40, 64, 1, 1, 1, BF16) == 1
