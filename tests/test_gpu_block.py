"""Rotary positions, the norms around a block and a whole differential block on the GPU against their 64-bit
definitions (reference64)."""
import pytest
import torch

import bi_level_routing_b200 as bra
import reference64 as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def randn(shape, seed, dtype=F32, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale + shift).to(dtype).cuda()


# ------------------------------------------------------------------ rotary positions

# B, H, W, heads, hd, n, axes: one token, heads turned whole and in part, pair counts of every access width
ROPE = [(1, 1, 1, 1, 32, 8, 2), (2, 7, 7, 2, 32, 8, 2), (1, 5, 9, 4, 20, 3, 2), (3, 4, 6, 2, 64, 8, 1), (2, 3, 3, 2, 12, 6, 1),
        (1, 13, 2, 4, 36, 4, 2), (1, 2, 2, 2, 128, 32, 2), (2, 6, 5, 2, 24, 1, 2), (1, 1, 70, 3, 16, 8, 1), (5, 3, 1, 8, 28, 2, 1)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shape", ROPE, ids=lambda s: "x".join(map(str, s)))
def test_rope(shape, layout, dtype):
    B, H, W, heads, hd, n, axes = shape
    q, k = (randn((B, H, W, heads * hd), s, dtype) for s in (1, 2))
    freqs, _ = bra.rope_frequencies(n, device="cuda")
    pos = torch.randint(0, 1 << 20, (B, H, W, axes), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    for origin, p, mscale, inverse in (((0, 0), None, 1.0, False), ((100000, 31), None, 1.2, True), ((0, 0), pos, 0.7, False),
                                       ((0, 0), -pos, 1.0, True)):
        got = bra.rope(q, k, freqs, heads, layout, axes, origin, p, mscale, inverse)
        for x, y in zip((q, k), got):
            want, tol = ref.rope(x, freqs, heads, layout, axes, origin, p, mscale, inverse)
            ref.check(y, want, tol, f"origin {origin} inverse {inverse}")
        # in place, and q alone
        q2, k2 = q.clone(), k.clone()
        bra.rope(q2, k2, freqs, heads, layout, axes, origin, p, mscale, inverse, q_out=q2, k_out=k2)
        assert torch.equal(q2, got[0]) and torch.equal(k2, got[1])
        alone = bra.rope(q, None, freqs, heads, layout, axes, origin, p, mscale, inverse)
        assert alone[1] is None and torch.equal(alone[0], got[0])


def test_rope_far_positions_and_not_finite():
    """Positions near 2^31 keep 64-bit angles; a NaN or an infinity stays in its own pair."""
    x = randn((1, 2, 3, 32), 4)
    freqs = torch.tensor([1.0, 0.37, 1e-4, 0.0], device="cuda")
    for origin in ((2 ** 31 - 5, -(2 ** 31)), (-12345678, 2 ** 30)):
        y, _ = bra.rope(x, None, freqs, 2, "half", 2, origin)
        want, tol = ref.rope(x, freqs, 2, "half", 2, origin, None, 1.0, False)
        ref.check(y, want, tol, f"origin {origin}")
    x[0, 1, 2, 3] = float("nan")
    y, _ = bra.rope(x, None, freqs, 2)
    assert int(torch.isnan(y).sum()) == 2 and bool(torch.isnan(y[0, 1, 2, 3])) and bool(torch.isnan(y[0, 1, 2, 7]))


def test_rope_inverse_is_the_gradient():
    """<rope(x), g> = <x, rope^-1(g)>: the inverse with the same mscale is the transpose, also against differences
    of the forward pass (linear: exact up to rounding)."""
    x, g = randn((2, 5, 4, 64), 5), randn((2, 5, 4, 64), 6)
    freqs, mscale = bra.rope_frequencies(8, scaling="yarn", factor=4.0, trained_extent=56, device="cuda")
    y, _ = bra.rope(x, None, freqs, 2, mscale=mscale)
    back, _ = bra.rope(g, None, freqs, 2, mscale=mscale, inverse=True)
    a, b = (y.double() * g.double()).sum(), (x.double() * back.double()).sum()
    # each product of the sums is off by at most 2^-21 of |x| |g| (mscale included)
    assert abs(float(a - b)) <= 2 * 2.0 ** -21 * mscale * float((x.double().norm() * g.double().norm()))
    e = torch.zeros_like(x)
    e.view(-1)[77] = 1.0
    y1, _ = bra.rope(x + e, None, freqs, 2, mscale=mscale)
    slope = ((y1 - y).double() * g.double()).sum()
    assert abs(float(slope - back.view(-1)[77])) <= 2.0 ** -20 * mscale * 64 * float(x.abs().max() + 1) * float(g.abs().max())


def test_rope_refusals():
    q = randn((1, 4, 4, 64), 7, BF16)
    f = torch.ones(8, device="cuda")
    both = torch.empty((2, 1, 4, 4, 64), dtype=BF16, device="cuda")
    for call in (lambda: bra.rope(q, q.float(), f, 2), lambda: bra.rope(q, None, f.double(), 2), lambda: bra.rope(q, None, f, 2, "whole"),
                 lambda: bra.rope(q, None, f, 2, pos=torch.zeros((1, 4, 4, 2), device="cuda")), lambda: bra.rope(q, None, f.cpu(), 2),
                 lambda: bra.rope(q, None, f, 2, k_out=q), lambda: bra.rope(q.cpu(), None, f, 2)):
        with pytest.raises(ValueError):
            call()
    shifted = both.view(-1)[8:8 + q.numel()].view(q.shape)
    for call in (lambda: bra.rope(q, None, torch.ones(9, device="cuda"), 2),          # 36 channels of 32
                 lambda: bra.rope(q, None, f, 3), lambda: bra.rope(q, None, f, 2, axes=3),
                 lambda: bra.rope(both[0], None, f, 2, q_out=shifted),                # outputs over a part of an input
                 lambda: bra.rope(q, both[0], f, 2, q_out=both[1], k_out=both[1]),
                 lambda: bra.rope(q, both[0], f, 2, q_out=both[0], k_out=both[1])):
        with pytest.raises(bra.BraError):
            call()


# ------------------------------------------------------------------ norms around a block

def norm_inputs(B, H, W, C, dtype, seed, gate, bias):
    g = {"none": None, "channel": randn((C,), seed + 1, scale=0.3, shift=0.6), "image": randn((B, C), seed + 1, scale=0.3, shift=0.6)}[gate]
    return dict(x=randn((B, H, W, C), seed + 2, dtype), h=randn((B, H, W, C), seed + 3, dtype, 0.7, 0.4), gate=g,
                post_weight=randn((C,), seed + 4, scale=0.2, shift=1.0), post_bias=randn((C,), seed + 5, scale=0.2) if bias else None,
                pre_weight=randn((C,), seed + 6, scale=0.2, shift=1.0), pre_bias=randn((C,), seed + 7, scale=0.2) if bias else None)


def plain(a, **kw):
    return ref.norm_residual(a["x"], a["h"], a["gate"], a["post_weight"], a["post_bias"], a["pre_weight"], a["pre_bias"], **kw)


def near(got, want, size, steps, what):
    """Within `steps` fp32 roundings (2^-24) of `size`, plus one rounding of got's type."""
    ref.check(got, want, torch.as_tensor(size, dtype=ref.F64).expand(want.shape) * steps * 2.0 ** -24, what)


def close(got, want, what):
    """The whole tensor: rounding the outputs moves each by at most half a step U of its value, so the difference's 2-norm is at most
    U times the result's; the fp32 arithmetic before it (some hundred steps of 2^-24 at most, mostly not in one
    direction) gets 2e-5 of it."""
    u = torch.finfo(got.dtype).eps / 2
    far = float((got.cpu().double() - want).norm()) / float(want.norm())
    assert far <= u + 2e-5, f"{what}: {far:.2e} of the result's norm"


def check_norms(a, alpha, eps, kind, with_ds=True):
    """Bounds. A mean of C values adds C roundings at most (trees add fewer), the mean of squares as many,
    so norm(h) is off by less than 2 C + 16 steps of its largest value + 1; s by that of |alpha x| + |gate p|.
    norm(s) divides by its deviation: errors of s count by r_s = 1 / sqrt(var + eps), as do those of the
    gradients by r_s and r_h. Each bound multiplies these magnitudes out."""
    C = a["x"].shape[-1]
    steps = 2 * C + 32
    s, y = bra.norm_residual(**a, alpha=alpha, eps=eps, kind=kind)
    want = plain(a, alpha=alpha, eps=eps, kind=kind)
    biggest = lambda t: 0.0 if t is None else float(t.abs().max())

    def spread(t):  # largest 1 / sqrt(var + eps) of rows
        t = t.double().cpu()
        m = t.var(-1, unbiased=False) if kind == "layer" else t.square().mean(-1)
        return float((m + eps).rsqrt().max())

    gate = 1.0 if a["gate"] is None else biggest(a["gate"])
    top = 0.0
    if a["h"] is not None:
        post = a["post_weight"] is not None
        rh = spread(a["h"]) if post else 1.0
        hn = (biggest(a["h"]) + 1) * max(rh, 1.0)
        p_size = hn * (biggest(a["post_weight"]) if post else 1.0) + biggest(a["post_bias"])
        top = gate * p_size
    s_size = abs(alpha) * biggest(a["x"]) + top
    if s is not None:
        near(s, want["s"], s_size, steps, "s")
        close(s, want["s"], "s")
    rs = max(spread(want["s"]), 1.0)
    if a["pre_weight"] is not None:
        near(y, want["y"], rs * 2 * s_size * biggest(a["pre_weight"]) + biggest(a["pre_bias"]), 2 * steps, "y")
        close(y, want["y"], "y")
    dy = randn(a["x"].shape, 91, a["x"].dtype) if a["pre_weight"] is not None else None
    ds = randn(a["x"].shape, 92, a["x"].dtype) if with_ds or dy is None else None
    grads = bra.norm_residual_backward(a["x"], a["h"], dy, ds, *(a[m] for m in ("gate", "post_weight", "post_bias", "pre_weight", "pre_bias")),
                                       alpha=alpha, eps=eps, kind=kind)
    want = plain(a, alpha=alpha, eps=eps, kind=kind, dy=dy, ds=ds)
    sn = 2 * rs * s_size  # bounds norm(s) + its error's factor
    dS = biggest(ds) + rs * biggest(dy) * biggest(a["pre_weight"]) * (2 + sn * sn)
    sizes = {"dx": abs(alpha) * dS}
    rows = a["x"].numel() // C
    if a["h"] is not None:
        dp = gate * dS
        sizes["dh"] = dp if not post else rh * dp * biggest(a["post_weight"]) * (2 + hn * hn)
        sizes.update(dgate=rows * dS * p_size, dpost_weight=rows * dp * hn, dpost_bias=rows * dp)
    sizes.update(dpre_weight=rows * biggest(dy) * sn, dpre_bias=rows * biggest(dy))
    for name in bra.NormGrads._fields:
        got = getattr(grads, name)
        if got is None:
            assert want.get(name) is None
            continue
        near(got, want[name], sizes[name], 4 * steps + (rows if name not in ("dx", "dh") else 0), name)
        close(got, want[name], name)


# C: one 16-byte vector, fewer threads than a warp, ragged vectors, one and several warps a row, the widest
WIDTHS = [8, 24, 64, 72, 128, 200, 256, 512, 520, 1000, 1024, 2048, 2056, 4096, 5000, 8192]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("C", WIDTHS)
def test_norm_widths(C, dtype):
    for kind, gate, bias, (B, H, W) in (("layer", "channel", True, (2, 3, 5)), ("rms", "image", False, (3, 7, 3))):
        check_norms(norm_inputs(B, H, W, C, dtype, C, gate, bias), 0.9, 1e-6, kind)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("absent", [("gate",), ("post_weight", "post_bias"), ("pre_weight", "pre_bias"), ("h", "gate", "post_weight", "post_bias"),
                                    ("post_bias",), ("pre_bias",), ("gate", "post_weight", "post_bias", "pre_bias")], ids="-".join)
def test_norm_parts(absent, dtype):
    for kind in ("layer", "rms"):
        a = norm_inputs(2, 5, 3, 64, dtype, 50, "image", True)
        a.update({name: None for name in absent})
        check_norms(a, 1.0, 1e-5, kind)
        check_norms(a, 0.5, 1e-5, kind, with_ds=False)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_norm_many_rows(dtype):
    """Enough rows that every CTA takes several and images end inside and between the CTAs' runs."""
    check_norms(norm_inputs(3, 71, 37, 64, dtype, 60, "image", True), 0.9, 1e-6, "layer")
    check_norms(norm_inputs(130, 3, 3, 128, dtype, 61, "image", False), 0.9, 1e-6, "rms")
    check_norms(norm_inputs(1, 101, 53, 264, dtype, 62, "channel", True), 0.9, 1e-6, "layer")


def test_norm_special_rows():
    """A constant row has norm 0 (eps keeps it finite); a row far from 0 keeps its deviation; one bad row stays
    one bad row; outputs may be the inputs' own buffers."""
    C = 64
    w = torch.ones(C, device="cuda")
    x = randn((1, 1, 6, C), 70)
    x[0, 0, 1] = 3.0
    x[0, 0, 2] += 1e4
    x[0, 0, 3, 5] = float("nan")
    x[0, 0, 4, 6] = float("inf")
    _, y = bra.norm_residual(x, pre_weight=w)
    want = torch.nn.functional.layer_norm(x.double(), (C,), eps=1e-6)
    ok = [0, 2, 5]
    # values near 1e4 carry 2^-24 1e4 themselves; the row's deviation is about 1
    assert float((y[0, 0, ok].double() - want[0, 0, ok]).abs().max()) <= 1e4 * C * 2.0 ** -24
    assert bool((y[0, 0, 1] == 0).all()) and bool(torch.isnan(y[0, 0, 3]).all()) and bool(torch.isnan(y[0, 0, 4, 6]))
    a = norm_inputs(2, 9, 5, 128, BF16, 71, "channel", True)
    s, y = bra.norm_residual(**a)
    b = {m: None if t is None else t.clone() for m, t in a.items()}
    bra.norm_residual(**b, s_out=b["x"], y_out=b["h"])
    assert torch.equal(b["x"], s) and torch.equal(b["h"], y)
    dy, ds = randn(s.shape, 72, BF16), randn(s.shape, 73, BF16)
    g = bra.norm_residual_backward(a["x"], a["h"], dy, ds, **{m: a[m] for m in a if m not in "xh"})
    dy2, ds2 = dy.clone(), ds.clone()
    g2 = bra.norm_residual_backward(a["x"], a["h"], dy2, ds2, **{m: a[m] for m in a if m not in "xh"}, dx=ds2, dh=dy2)
    assert all(torch.equal(u, v) for u, v in zip(g, g2))


def test_norm_refusals():
    a = norm_inputs(2, 3, 4, 64, BF16, 80, "image", True)
    for change in (dict(h=a["h"].float()), dict(gate=a["gate"][:1].contiguous()), dict(post_weight=a["post_weight"].bfloat16()),
                   dict(kind="batch"), dict(pre_weight=a["pre_weight"].cpu()), dict(pre_weight=None, pre_bias=None, y_out=a["x"])):
        with pytest.raises(ValueError):
            bra.norm_residual(**{**a, **change})
    for change in (dict(post_weight=None), dict(pre_weight=None), dict(h=None), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(s_out=a["x"], y_out=a["x"])):
        with pytest.raises(bra.BraError):
            bra.norm_residual(**{**a, **change})
    wide = randn((1, 1, 1, 8200), 81, BF16)
    with pytest.raises(bra.BraError):
        bra.norm_residual(wide, pre_weight=torch.ones(8200, device="cuda"))


# ------------------------------------------------------------------ the block

@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
def test_block_and_its_gradients(captured):
    """One differential block, y = norm(x), q = rope(y w_q), k = rope(y w_k), v = y w_v, routed differential
    attention, s = x + gate norm(attention), and back to x, against automatic differentiation in 64 bits of the same
    steps with the routing fixed. fp32 all through, so that only fp32 roundings part them: the chain's gain on
    an error stays below 1e4 here (five steps that each add a few hundred roundings of values below 10)."""
    B, H, W, C, heads, n_win, topk = 2, 12, 12, 64, 1, 3, 2
    x = randn((B, H, W, C), 100)
    w = [randn((C, C), 101 + i, scale=C ** -0.5) for i in range(3)]
    n1, n2, gate = (randn((C,), 110 + i, scale=0.1, shift=1.0) for i in range(3))
    lam = torch.tensor([0.4], device="cuda")
    freqs, _ = bra.rope_frequencies(8, device="cuda")
    g = randn((B, H, W, C), 120)

    def step():
        _, y = bra.norm_residual(x, pre_weight=n1)
        q, k, v = (y @ m for m in w)
        qr, kr = bra.rope(q, k, freqs, 2 * heads)
        out, idx = bra.forward_diff(qr, kr, v, lam, n_win, topk, heads)
        s, _ = bra.norm_residual(x, out, gate=gate, post_weight=n2)
        tail = bra.norm_residual_backward(x, out, None, g, gate=gate, post_weight=n2)
        dqr, dkr, dv, dlam = bra.diff_attend_backward(qr, kr, v, idx, lam, tail.dh, heads, n_win)
        dq, dk = bra.rope(dqr, dkr, freqs, 2 * heads, inverse=True)
        dy = dq @ w[0].T + dk @ w[1].T + dv @ w[2].T
        head = bra.norm_residual_backward(x, None, dy, None, pre_weight=n1)
        return s, idx, tail.dx + head.dx, dlam, tail.dgate, tail.dpost_weight, head.dpre_weight

    got = step()
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = step()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, held))
        got = held
    s, idx, dx, dlam, dgate, dn2, dn1 = got
    D = lambda t: t.double().cpu().requires_grad_(True)
    x6, lam6, gate6, n26, n16 = map(D, (x, lam, gate, n2, n1))
    y = torch.nn.functional.layer_norm(x6, (C,), eps=1e-6) * n16
    ang = torch.stack(torch.meshgrid(torch.arange(H), torch.arange(W), indexing="ij"), -1)[:, :, None, :, None] * freqs.double().cpu()

    def turn(t):
        t = t.view(B, H, W, 2 * heads, 2, 2, 8)
        a, b, c, s_ = t[..., 0, :], t[..., 1, :], torch.cos(ang), torch.sin(ang)
        return torch.stack((a * c - b * s_, b * c + a * s_), -2).reshape(B, H, W, C)

    q, k, v = (y @ m.double().cpu() for m in w)
    q, k = turn(q), turn(k)
    tok = ref.region_tokens(H, W, n_win)
    out = torch.zeros(B, H * W, C, dtype=ref.F64)
    for b in range(B):
        for r, t in enumerate(tok):
            src = torch.cat([tok[int(i)] for i in idx[b, r]])
            f = lambda z, at: z[b].reshape(H * W, C)[at]
            p = [torch.softmax(f(q, t)[:, i] @ f(k, src)[:, i].T / 32 ** 0.5, -1) for i in (slice(0, 32), slice(32, 64))]
            out = out.index_put((torch.tensor(b), t), (p[0] - lam6[0] * p[1]) @ f(v, src))
    s6 = x6 + gate6 * torch.nn.functional.layer_norm(out.view(B, H, W, C), (C,), eps=1e-6) * n26
    (s6 * g.double().cpu()).sum().backward()
    for name, a, b in (("s", s, s6.detach()), ("dx", dx, x6.grad), ("dlam", dlam, lam6.grad), ("dgate", dgate, gate6.grad),
                       ("post weight", dn2, n26.grad), ("pre weight", dn1, n16.grad)):
        err = float((a.double().cpu() - b).abs().max())
        assert err <= 1e4 * 2.0 ** -24 * max(1.0, float(b.abs().max())), f"{name}: {err}"


# ------------------------------------------------------------------ calls at the edges

@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_empty_batches(dtype):
    """No image: empty results, and sums over nothing are 0."""
    x = torch.empty((0, 6, 6, 64), device="cuda", dtype=dtype)
    idx = torch.empty((0, 9, 2), device="cuda", dtype=torch.int32)
    lam, w = torch.ones(2, device="cuda"), torch.ones(64, device="cuda")
    assert bra.diff_attend(x, x, x, idx, lam, 2, 3).shape == x.shape
    out, routed = bra.forward_diff(x, x, x, lam, 3, 2, 2)
    assert out.shape == x.shape and routed.shape == idx.shape
    grads = bra.diff_attend_backward(x, x, x, idx, lam, x, 2, 3)
    assert all(t.shape == x.shape for t in grads[:3]) and grads[3].tolist() == [0.0, 0.0]
    q, k = bra.rope(x, x, torch.ones(4, device="cuda"), 2)
    assert q.shape == x.shape and k.shape == x.shape
    for gate in (w, torch.empty((0, 64), device="cuda")):
        s, y = bra.norm_residual(x, x, gate=gate, post_weight=w, post_bias=w, pre_weight=w)
        assert s.shape == x.shape and y.shape == x.shape
        g = bra.norm_residual_backward(x, x, x, x, gate=gate, post_weight=w, post_bias=w, pre_weight=w)
        assert g.dx.shape == x.shape and g.dh.shape == x.shape and g.dgate.shape == gate.shape
        assert all(not bool(t.any()) for t in (g.dgate, g.dpost_weight, g.dpost_bias, g.dpre_weight))


def test_two_threads():
    """Two threads, each on a stream of its own, get what they get one after the other."""
    import threading

    def inputs(seed):
        q, k, v, d = (randn((3, 20, 20, 64), seed + i, BF16) for i in range(4))
        idx = torch.randint(0, 4, (3, 4, 2), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()
        return q, k, v, d, idx, randn((2,), seed + 5), randn((64,), seed + 6)

    freqs, _ = bra.rope_frequencies(4, device="cuda")

    def work(q, k, v, d, idx, lam, w):
        q, k = bra.rope(q, k, freqs, 4)
        out = bra.diff_attend(q, k, v, idx, lam, 2, 2)
        s, y = bra.norm_residual(v, out, gate=w, post_weight=w, pre_weight=w)
        n = bra.norm_residual_backward(v, out, d, None, gate=w, post_weight=w, pre_weight=w)
        return [s, y, *(t for t in n if t is not None), *bra.diff_attend_backward(q, k, v, idx, lam, n.dh, 2, 2)]

    sets = [inputs(300), inputs(400)]
    want = [work(*s) for s in sets]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(30):
                    got = work(*sets[i])
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        wrong.append(i)
        except Exception as e:  # noqa: BLE001  (reported below: a thread's exception ends nothing)
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# (elements just above 2^32 in bf16, above 2^31 in fp32) regions of 1024, 64 and 4 tokens; 64-token regions, two routed
FAR = [(33, 1024, 128, 32, 1, BF16), (2080, 128, 128, 16, 1, BF16), (2080, 128, 128, 16, 2, BF16), (33000, 32, 128, 16, 3, BF16),
       (1050, 128, 128, 16, 1, F32)]


@pytest.mark.parametrize("B,H,C,n_win,topk,dtype", FAR, ids=lambda v: str(v).removeprefix("torch."))
def test_offsets_past_32_bits(B, H, C, n_win, topk, dtype):
    """The last images of arrays whose offsets pass 32 bits are those of a call on these images alone, bit for bit."""
    assert B * H * H * C > (2 ** 32 if dtype is BF16 else 2 ** 31)
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 70e9:
        pytest.skip("needs 70 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty((B, H, H, C), device="cuda", dtype=dtype)
    for part in x.split(max(1, B // 16)):
        part.normal_(generator=gen)
    R = n_win * n_win
    idx = torch.randint(0, R, (B, R, topk), generator=gen, device="cuda", dtype=torch.int32)
    lam, w = torch.full((1,), 0.3, device="cuda"), torch.rand(C, generator=gen, device="cuda")
    tail = x[-2:].clone()
    last = idx[-2:].contiguous()
    same = lambda far, near: torch.equal(far[-2:], near)
    far = bra.diff_attend(x, x, x, idx, lam, 1, n_win)
    assert same(far, bra.diff_attend(tail, tail, tail, last, lam, 1, n_win))
    del far
    far = bra.diff_attend_backward(x, x, x, idx, lam, x, 1, n_win)
    near = bra.diff_attend_backward(tail, tail, tail, last, lam, tail, 1, n_win)
    assert all(same(a, b) for a, b in zip(far[:3], near[:3]))
    del far
    freqs, _ = bra.rope_frequencies(16, device="cuda")
    far = bra.rope(x, None, freqs, 2)[0]
    assert same(far, bra.rope(tail, None, freqs, 2)[0])
    del far
    s, y = bra.norm_residual(x, x, gate=w, post_weight=w, pre_weight=w)
    near = bra.norm_residual(tail, tail, gate=w, post_weight=w, pre_weight=w)
    assert same(s, near[0]) and same(y, near[1])
    del s, y
    far = bra.norm_residual_backward(x, x, x, x, gate=w, post_weight=w, pre_weight=w)
    near = bra.norm_residual_backward(tail, tail, tail, tail, gate=w, post_weight=w, pre_weight=w)
    assert same(far.dx, near.dx) and same(far.dh, near.dh)
    assert bra.check_device_error() == 0
    del far
    torch.cuda.empty_cache()
