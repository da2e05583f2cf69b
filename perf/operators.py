"""Performance cases of the differential block: differential attention over routed regions and its
gradients, rotary positions of q and k, and the norms around a block with its gate and residual.

Each case is one pass through one operator. `run` takes it through elementary torch operations in
32 bits (64 for angles and column sums), or, where `own` is true, through the package's calls.
`exact` computes the same from the definitions in 64 bits.

Definitions. Feature maps are [B, H, W, C], cut into n_win x n_win regions numbered row by row.
  diff_attend   head h owns hd = C / heads channels; the first hd / 2 of its q and k make map 1,
                the others map 2. Over the tokens of the regions idx[b, r, :], for a query of region
                r: out = (softmax(s q1 k1^T) - lam[h] softmax(s q2 k2^T)) v, s = (hd / 2)^-1/2.
  diff_backward the gradients of sum(dout * out) by q, k, v and lam.
  rope          the first 2 axes n channels of each head hold `axes` blocks of n pairs, block a
                turned by position[a] * freqs[i] and scaled by mscale; the others are unchanged.
                Pair i is (2 i, 2 i + 1) or (i, i + n). `inverse` turns back (the backward pass).
  norm          s = alpha x + gate * (norm(h) w_post + b_post), y = norm(s) w_pre + b_pre.
  norm_backward the gradients of sum(ds * s) + sum(dy * y) by x, h, gate and the weights.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _attn(name, op, B, hr, wr, n_win, topk, heads, hd, dtype):
    return {"name": name, "op": op, "B": B, "H": hr * n_win, "W": wr * n_win, "n_win": n_win, "topk": topk,
            "heads": heads, "hd": hd, "dtype": dtype}


def _rope(name, B, H, W, heads, hd, n, axes, layout, dtype, far=0, given=False, inverse=False):
    return {"name": name, "op": "rope", "B": B, "H": H, "W": W, "heads": heads, "hd": hd, "n": n, "axes": axes,
            "layout": layout, "dtype": dtype, "far": far, "given": given, "inverse": inverse}


def _norm(name, op, B, H, W, C, kind, gate, bias, dtype):
    return {"name": name, "op": op, "B": B, "H": H, "W": W, "C": C, "kind": kind, "gate": gate, "bias": bias,
            "dtype": dtype}


def listed():
    return [
        # one image through a last-stage block: 49 one-token regions, every region routed; latency
        _attn("diff_stage4_one_image", "diff_attend", 1, 1, 1, 7, 49, 8, 64, "bf16"),
        # a batch through a first-stage block: 64-token regions, one routed region
        _attn("diff_stage1", "diff_attend", 64, 8, 8, 7, 1, 1, 64, "bf16"),
        # global attention over a 128 x 128 map (one region): 16384 tokens, the long end
        _attn("diff_global_highres", "diff_attend", 2, 128, 128, 1, 1, 2, 64, "bf16"),
        # odd windows (9 x 7 tokens) and a head of 48 channels in fp32
        _attn("diff_odd_f32", "diff_attend", 4, 9, 7, 5, 3, 2, 48, "f32"),
        # a training step's backward of a second-stage block: 16-token regions, four routed
        _attn("diff_backward_stage2", "diff_backward", 64, 4, 4, 7, 4, 2, 64, "bf16"),
        # backward of global attention over a 64 x 64 map with 128-channel heads
        _attn("diff_backward_global", "diff_backward", 4, 64, 64, 1, 1, 4, 128, "bf16"),
        # q and k of a first-stage batch, before routing
        _rope("rope_stage1", 64, 56, 56, 2, 32, 8, 2, "half", "bf16"),
        # the way back for fp32 gradients: raster positions handed in, part of the head, adjacent pairs
        _rope("rope_backward_partial_f32", 8, 128, 128, 2, 32, 8, 1, "interleaved", "f32", far=100000, given=True,
              inverse=True),
        # one image at the last stage: latency
        _norm("norm_stage4_one_image", "norm", 1, 7, 7, 512, "layer", "channel", True, "bf16"),
        # a first-stage batch: short rows, many of them
        _norm("norm_stage1", "norm", 64, 56, 56, 64, "layer", "channel", True, "bf16"),
        # backward of a second-stage batch, with a gate of its own for each image
        _norm("norm_backward_stage2", "norm_backward", 64, 28, 28, 128, "layer", "image", True, "bf16"),
        # backward of wide rows without biases, as in a long sequence model
        _norm("norm_backward_wide", "norm_backward", 4, 64, 32, 4096, "rms", "channel", False, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above."""
    op = rng.choice(["diff_attend", "diff_attend", "diff_backward", "diff_backward", "rope", "norm", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("diff_attend", "diff_backward"):
        hd = rng.choice([8, 16, 24, 32, 40, 48, 64, 64, 80, 96, 112, 128, 128])
        heads = rng.choice([1, 2, 3, 4, 8])
        n_win = rng.choice([1, 1, 2, 3, 5, 7, 7, 8, 14, 16])
        hr, wr = (_log_int(rng, 1, max(1, 96 // n_win)) for _ in range(2))
        R = n_win * n_win
        topk = min(R, _log_int(rng, 1, R))
        # query-key pairs times channels; fp32 maps, which run at a fraction of the speed, are drawn smaller
        most = 2e10 if dtype == "bf16" else 2e9
        while R * topk * (hr * wr) ** 2 * heads * hd > most:
            hr, wr = (hr + 1) // 2, wr
            if hr == 1:
                hr, wr = wr, hr
        N = hr * wr * R
        B = min(_log_int(rng, 1, 64), int(most / (N * topk * hr * wr * heads * hd)),
                int((2.5e7 if dtype == "bf16" else 1.2e7) / (N * heads * hd)))
        B = max(1, B)
        return {k: v for k, v in _attn("", op, B, hr, wr, n_win, topk, heads, hd, dtype).items() if k != "name"}
    if op == "rope":
        hd = 4 * rng.randint(1, 32)
        axes = rng.choice([1, 2])
        n = max(1, int(hd * rng.choice([0.25, 0.5, 1.0])) // (2 * axes))
        heads = 2 * rng.randint(1, 8)
        H, W = _log_int(rng, 1, 130), _log_int(rng, 1, 130)
        B = max(1, min(_log_int(rng, 1, 64), int(1.2e7 / (H * W * heads * hd))))
        given = rng.random() < 0.4
        c = _rope("", B, H, W, heads, hd, n, axes, rng.choice(["half", "interleaved"]), dtype,
                  far=rng.choice([0, 0, 1000, 1000000]), given=given, inverse=rng.random() < 0.5)
        return {k: v for k, v in c.items() if k != "name"}
    C = 8 * _log_int(rng, 1, 1024)
    rows = max(1, min(_log_int(rng, 1, 200000), int((3e7 if dtype == "bf16" else 1.5e7) / C)))
    B = rng.choice([1, 2, 3, 8])
    H = max(1, int(math.sqrt(rows / B)))
    W = max(1, rows // (B * H))
    kind = rng.choice(["layer", "rms"])
    c = _norm("", op, B, H, W, C, kind, rng.choice(["none", "channel", "image"]), kind == "layer" and rng.random() < 0.7,
              dtype)
    return {k: v for k, v in c.items() if k != "name"}


# ------------------------------------------------------------------ inputs

ALPHA, EPS, MSCALE = 0.9, 1e-6, 1.1


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    st = dict(case)
    if case["op"] in ("diff_attend", "diff_backward"):
        B, H, W, n, heads = case["B"], case["H"], case["W"], case["n_win"], case["heads"]
        C, R = heads * case["hd"], n * n

        def feature():  # tokens around their region's offset, so that regions differ
            off = 0.5 * normal(B, n, 1, n, 1, C)
            return (normal(B, n, H // n, n, W // n, C) + off).reshape(B, H, W, C).to(dt)

        st.update(q=feature(), k=feature(), v=feature(), dout=normal(B, H, W, C).to(dt))
        st["lam"] = 0.2 + 0.6 * torch.rand(heads, generator=g, device="cuda")
        order = torch.rand((B, R, R), generator=g, device="cuda").argsort(dim=-1)  # distinct regions a row
        st["idx"] = order[:, :, :case["topk"]].to(torch.int32).contiguous()
        return st
    B, H, W = case["B"], case["H"], case["W"]
    if case["op"] == "rope":
        C = case["heads"] * case["hd"]
        st.update(q=normal(B, H, W, C).to(dt), k=normal(B, H, W, C).to(dt))
        i = torch.arange(case["n"], device="cuda", dtype=torch.float64)
        st["freqs"] = (10000.0 ** (-i / case["n"])).float()
        st["pos"] = None
        if case["given"]:  # crops and packed maps: a position for each token
            p = torch.randint(0, max(W, H, case["far"]), (B, H, W, case["axes"]), generator=g, device="cuda")
            st["pos"] = p.to(torch.int32)
        return st
    C = case["C"]
    st.update(x=normal(B, H, W, C).to(dt), h=(0.7 * normal(B, H, W, C) + 0.3).to(dt))
    st["gate"] = {"none": None, "channel": 0.5 + 0.2 * normal(C), "image": 0.5 + 0.2 * normal(B, C)}[case["gate"]]
    st["w_post"], st["w_pre"] = 1 + 0.1 * normal(C), 1 + 0.1 * normal(C)
    st["b_post"], st["b_pre"] = (0.1 * normal(C), 0.1 * normal(C)) if case["bias"] else (None, None)
    if case["op"] == "norm_backward":
        st.update(dy=normal(B, H, W, C).to(dt), ds=normal(B, H, W, C).to(dt))
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _run_own(st)
    return {"diff_attend": _diff, "diff_backward": _diff_backward, "rope": _rope_plain, "norm": _norm_plain,
            "norm_backward": _norm_backward}[st["op"]](st)


def _run_own(st):
    import bi_level_routing_b200 as bra

    op = st["op"]
    if op == "diff_attend":
        return bra.diff_attend(st["q"], st["k"], st["v"], st["idx"], st["lam"], st["heads"], st["n_win"])
    if op == "diff_backward":
        return bra.diff_attend_backward(st["q"], st["k"], st["v"], st["idx"], st["lam"], st["dout"], st["heads"],
                                        st["n_win"])
    if op == "rope":
        return bra.rope(st["q"], st["k"], st["freqs"], st["heads"], layout=st["layout"], axes=st["axes"],
                        origin=(st["far"], st["far"]), pos=st["pos"], mscale=MSCALE, inverse=st["inverse"])
    kw = dict(gate=st["gate"], post_weight=st["w_post"], post_bias=st["b_post"], pre_weight=st["w_pre"],
              pre_bias=st["b_pre"], alpha=ALPHA, eps=EPS, kind=st["kind"])
    if op == "norm":
        return bra.norm_residual(st["x"], st["h"], **kw)
    grads = bra.norm_residual_backward(st["x"], st["h"], st["dy"], st["ds"], **kw)
    return [t for t in grads if t is not None]


# The plain forms: elementary operations in 32 bits, rounded once at the end.

def _to_regions(x, n):
    """[B, H, W, C] -> [B, R, tokens, C]."""
    B, H, W, C = x.shape
    return x.view(B, n, H // n, n, W // n, C).permute(0, 1, 3, 2, 4, 5).reshape(B, n * n, (H // n) * (W // n), C)


def _from_regions(x, n, H, W):
    B, C = x.shape[0], x.shape[-1]
    return x.view(B, n, n, H // n, W // n, C).permute(0, 1, 3, 2, 4, 5).reshape(B, H, W, C)


def _pieces(st):
    """(image, head, first region, last region, first query, last query) of pieces whose score
    matrices hold at most 2^28 elements."""
    R, rs = st["n_win"] ** 2, (st["H"] // st["n_win"]) * (st["W"] // st["n_win"])
    keys = st["topk"] * rs
    rows = max(1, 2 ** 28 // keys)
    images = max(1, min(rows // (R * rs * st["heads"]), 2 ** 29 // (R * keys * st["heads"] * st["hd"])))
    if R * rs * st["heads"] <= rows:
        return [(slice(b, b + images), slice(None), slice(None)) for b in range(0, st["B"], images)]
    return [(slice(b, b + 1), slice(r, r + 1), slice(t, t + max(1, rows // st["heads"])))
            for b in range(st["B"]) for r in range(R) for t in range(0, rs, max(1, rows // st["heads"]))]


def _maps(st, qr, kr, vr, piece):
    """Of one piece: the queries' two maps p1, p2 [b, r, heads, t, keys] and what they were made of."""
    b, r, t = piece
    heads, hd = st["heads"], st["hd"]
    q = qr[b, r][:, :, t].float()
    B, nr, nt, _ = q.shape
    idx = st["idx"][b, r].long()
    at = torch.arange(B, device=q.device).view(B, 1, 1)
    k = kr[b][at, idx].flatten(2, 3).float()
    v = vr[b][at, idx].flatten(2, 3).float()
    q = q.view(B, nr, nt, heads, 2, hd // 2).permute(4, 0, 1, 3, 2, 5)
    k = k.view(B, nr, -1, heads, 2, hd // 2).permute(4, 0, 1, 3, 2, 5)
    v = v.view(B, nr, -1, heads, hd).transpose(2, 3)
    scale = (hd // 2) ** -0.5
    p1 = torch.softmax((q[0] @ k[0].transpose(-1, -2)) * scale, -1)
    p2 = torch.softmax((q[1] @ k[1].transpose(-1, -2)) * scale, -1)
    return q, k, v, p1, p2, idx, scale


def _diff(st):
    n, H, W = st["n_win"], st["H"], st["W"]
    qr, kr, vr = (_to_regions(st[x], n) for x in "qkv")
    out = torch.empty_like(qr)
    lam = st["lam"].view(1, 1, -1, 1, 1)
    for piece in _pieces(st):
        _, _, v, p1, p2, _, _ = _maps(st, qr, kr, vr, piece)
        o = (p1 - lam * p2) @ v
        b, r, t = piece
        out[b, r, t] = o.transpose(2, 3).flatten(3).to(out.dtype)
    return _from_regions(out, n, H, W)


def _diff_backward(st):
    n, H, W, heads = st["n_win"], st["H"], st["W"], st["heads"]
    qr, kr, vr, gr = (_to_regions(st[x], n) for x in ("q", "k", "v", "dout"))
    B, R, rs, C = qr.shape
    dq = torch.empty(qr.shape, device=qr.device)
    dk, dv = torch.zeros_like(dq), torch.zeros_like(dq)
    dlam = torch.zeros(heads, device=qr.device, dtype=torch.float64)
    lam = st["lam"].view(1, 1, -1, 1, 1)
    for piece in _pieces(st):
        q, k, v, p1, p2, idx, scale = _maps(st, qr, kr, vr, piece)
        b, r, t = piece
        do = gr[b, r][:, :, t].float().unflatten(-1, (heads, -1)).transpose(2, 3)
        dp = do @ v.transpose(-1, -2)
        gv = (p1 - lam * p2).transpose(-1, -2) @ do
        d1, d2 = (p1 * dp).sum(-1, keepdim=True), (p2 * dp).sum(-1, keepdim=True)
        dlam -= d2.sum((0, 1, 3, 4), dtype=torch.float64)
        s1, s2 = p1 * (dp - d1) * scale, -lam * p2 * (dp - d2) * scale
        gq = torch.stack((s1 @ k[0], s2 @ k[1]), -2)  # [b, r, heads, t, 2, d]
        dq[b, r, t] = gq.transpose(2, 3).flatten(3)
        gk = torch.stack((s1.transpose(-1, -2) @ q[0], s2.transpose(-1, -2) @ q[1]), -2).transpose(2, 3).flatten(3)
        nb = idx.shape[0]
        rows = (torch.arange(nb, device=idx.device).view(nb, 1, 1) * R + idx).flatten()
        for whole, part in ((dk, gk), (dv, gv.transpose(2, 3).flatten(3))):
            whole[b].view(nb * R, rs, C).index_add_(0, rows, part.reshape(-1, rs, C))
    dt = qr.dtype
    return tuple(_from_regions(x, n, H, W).to(dt) for x in (dq, dk, dv)) + (dlam.float(),)


def _angles(st):
    """Angles [B or 1, H, W, 1, axes, n] in 64 bits."""
    H, W, axes = st["H"], st["W"], st["axes"]
    f = st["freqs"].double()
    if st["pos"] is not None:
        pos = st["pos"].double()
    else:
        y = torch.arange(H, device=f.device, dtype=torch.float64).view(H, 1)
        x = torch.arange(W, device=f.device, dtype=torch.float64).view(1, W)
        if axes == 2:
            pos = torch.stack(((y + st["far"]).expand(H, W), (x + st["far"]).expand(H, W)), -1)
        else:
            pos = ((y + st["far"]) * W + x + st["far"]).unsqueeze(-1)
        pos = pos.unsqueeze(0)
    return pos[:, :, :, None, :, None] * f


def _rope_plain(st):
    ang = _angles(st)
    cos, sin = torch.cos(ang).float() * MSCALE, torch.sin(ang).float() * MSCALE
    if st["inverse"]:
        sin = -sin
    n, axes, hd = st["n"], st["axes"], st["hd"]
    rot = 2 * axes * n
    outs = []
    for x in (st["q"], st["k"]):
        h = x.float().unflatten(-1, (st["heads"], hd))
        r = h[..., :rot].unflatten(-1, (axes, 2 * n))
        if st["layout"] == "half":
            a, b = r[..., :n], r[..., n:]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        outs.append(torch.cat((turned.flatten(-2), h[..., rot:]), -1).flatten(-2).to(x.dtype))
    return tuple(outs)


def _statistics(z, kind):
    """The normalised rows and their factor 1 / sqrt(variance + eps)."""
    if kind == "layer":
        z = z - z.mean(-1, keepdim=True)
    r = torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS)
    return z * r, r


def _gate(st):
    g = st["gate"]
    return 1.0 if g is None else g if g.dim() == 1 else g[:, None, None, :]


def _norm_plain(st):
    hn, _ = _statistics(st["h"].float(), st["kind"])
    p = hn * st["w_post"]
    if st["b_post"] is not None:
        p = p + st["b_post"]
    s = ALPHA * st["x"].float() + _gate(st) * p
    y = _statistics(s, st["kind"])[0] * st["w_pre"]
    if st["b_pre"] is not None:
        y = y + st["b_pre"]
    return s.to(st["x"].dtype), y.to(st["x"].dtype)


def _norm_backward(st):
    kind, gate = st["kind"], _gate(st)
    hn, rh = _statistics(st["h"].float(), kind)
    p = hn * st["w_post"]
    if st["b_post"] is not None:
        p = p + st["b_post"]
    sn, rs = _statistics(ALPHA * st["x"].float() + gate * p, kind)

    def back(up, z, r):
        up = up - z * (up * z).mean(-1, keepdim=True)
        return r * (up - up.mean(-1, keepdim=True) if kind == "layer" else up)

    def column(t, dims=(0, 1, 2)):
        return t.sum(dims, dtype=torch.float64).float()

    dy = st["dy"].float()
    ds = st["ds"].float() + back(dy * st["w_pre"], sn, rs)
    dp = gate * ds
    dh = back(dp * st["w_post"], hn, rh)
    dt = st["x"].dtype
    out = [(ALPHA * ds).to(dt), dh.to(dt)]
    if st["gate"] is not None:
        out.append(column(ds * p) if st["gate"].dim() == 1 else column(ds * p, (1, 2)))
    out.append(column(dp * hn))
    if st["b_post"] is not None:
        out.append(column(dp))
    out.append(column(dy * sn))
    if st["b_pre"] is not None:
        out.append(column(dy))
    return out


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    if case["op"] in ("diff_attend", "diff_backward"):
        rs = case["H"] * case["W"] // case["n_win"] ** 2
        pairs = case["B"] * case["H"] * case["W"] * case["topk"] * rs * case["heads"] * case["hd"]
        if pairs > 1.5e11:
            return None
    st = prepare(case, seed)
    if case["op"] in ("diff_attend", "diff_backward"):
        return _exact_diff(st)
    if case["op"] == "rope":
        return _exact_rope(st)
    return _exact_norm(st)


def _window_tokens(st):
    """[R, tokens] flat y * W + x of each region's tokens, row by row."""
    n, H, W = st["n_win"], st["H"], st["W"]
    grid = torch.arange(H * W, device="cuda").view(H, W)
    return torch.stack([w.reshape(-1) for rows in grid.chunk(n, 0) for w in rows.chunk(n, 1)])


def _exact_diff(st):
    """Head by head, a few images (or a run of queries) at a time; the gradients by automatic
    differentiation of the definition."""
    B, H, W, heads, hd = st["B"], st["H"], st["W"], st["heads"], st["hd"]
    d, N = hd // 2, H * W
    tok = _window_tokens(st)
    R, rs = tok.shape
    keys = st["topk"] * rs
    want = st["op"] == "diff_backward"
    x = {m: st[m].double().view(B, N, heads, hd) for m in ("q", "k", "v", "dout")}
    out = torch.zeros_like(x["q"])
    grad = {m: torch.zeros_like(x[m]) for m in "qkv"}
    dlam = torch.zeros(heads, device="cuda", dtype=torch.float64)
    most = 2 ** 25
    nb = max(1, min(B, most // (R * rs * keys), 2 ** 27 // (R * keys * hd)))
    nq = max(1, min(rs, most // (R * keys))) if nb == 1 else rs
    for h in range(heads):
        for b0 in range(0, B, nb):
            bs = slice(b0, min(B, b0 + nb))
            src = tok[st["idx"][bs].long()].flatten(2)  # [b, R, keys] tokens routed to
            bb = torch.arange(src.shape[0], device="cuda").view(-1, 1, 1)
            for t0 in range(0, rs, nq):
                mine = tok[:, t0:t0 + nq]
                q, k, v = (x[m][bs, :, h].clone().requires_grad_(want) for m in "qkv")
                lam = st["lam"][h].double().clone().requires_grad_(want)
                with torch.set_grad_enabled(want):
                    qq, kk, vv = q[:, mine], k[bb, src], v[bb, src]
                    maps = [torch.softmax(torch.einsum("brtc,brjc->brtj", qq[..., i], kk[..., i]) / math.sqrt(d), -1)
                            for i in (slice(0, d), slice(d, hd))]
                    o = torch.einsum("brtj,brjc->brtc", maps[0] - lam * maps[1], vv)
                    if want:
                        (o * x["dout"][bs, :, h][:, mine]).sum().backward()
                        for m, t in zip("qkv", (q, k, v)):
                            grad[m][bs, :, h] += t.grad
                        dlam[h] += lam.grad
                    else:
                        out[bs, mine.flatten(), h] = o.flatten(1, 2)
    if want:
        return tuple(grad[m].view(B, H, W, -1) for m in "qkv") + (dlam,)
    return out.view(B, H, W, -1)


def _exact_rope(st):
    """As a product of complex numbers."""
    n, axes, heads, hd = st["n"], st["axes"], st["heads"], st["hd"]
    ang = _angles(st)
    turn = torch.polar(torch.full_like(ang, MSCALE), -ang if st["inverse"] else ang)
    outs = []
    for x in (st["q"], st["k"]):
        full = x.double().view(*x.shape[:3], heads, hd).clone()
        for a in range(axes):
            c0 = 2 * n * a
            first, second = ((slice(c0, c0 + n), slice(c0 + n, c0 + 2 * n)) if st["layout"] == "half" else
                             (slice(c0, c0 + 2 * n, 2), slice(c0 + 1, c0 + 2 * n, 2)))
            z = torch.complex(full[..., first], full[..., second]) * turn[..., a, :]
            full[..., first], full[..., second] = z.real, z.imag
        outs.append(full.view(x.shape))
    return tuple(outs)


def _exact_norm(st):
    def leaf(name):
        t = st.get(name)
        return None if t is None else t.double().requires_grad_(st["op"] == "norm_backward")

    names = ("x", "h", "gate", "w_post", "b_post", "w_pre", "b_pre")
    x, h, gate, w_post, b_post, w_pre, b_pre = leaves = [leaf(m) for m in names]

    def norm(z):
        if st["kind"] == "layer":
            return (z - z.mean(-1, keepdim=True)) / torch.sqrt(z.var(-1, unbiased=False, keepdim=True) + EPS)
        return z / torch.sqrt(z.square().mean(-1, keepdim=True) + EPS)

    p = norm(h) * w_post + (0 if b_post is None else b_post)
    g = 1 if gate is None else gate if gate.dim() == 1 else gate.view(gate.shape[0], 1, 1, -1)
    s = ALPHA * x + g * p
    y = norm(s) * w_pre + (0 if b_pre is None else b_pre)
    if st["op"] == "norm":
        return s, y
    ((s * st["ds"].double()).sum() + (y * st["dy"].double()).sum()).backward()
    return [t.grad for t in leaves if t is not None]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("diff_attend", "diff_backward"):
        n, heads, hd = case["n_win"], case["heads"], case["hd"]
        tokens = case["B"] * case["H"] * case["W"]
        keys = case["topk"] * (case["H"] // n) * (case["W"] // n)
        side = 4 * case["B"] * n * n * case["topk"] + 4 * heads
        pair = 2 * tokens * keys * heads * hd  # one product over a head's channels, all pairs
        if case["op"] == "diff_attend":  # two half-head score products and one with the values
            return {"bytes": 4 * tokens * heads * hd * e + side, "flops": 2 * pair}
        return {"bytes": 7 * tokens * heads * hd * e + side + 4 * heads, "flops": 5 * pair}
    tokens = case["B"] * case["H"] * case["W"]
    if case["op"] == "rope":
        given = 4 * tokens * case["axes"] if case["given"] else 0
        return {"bytes": 4 * tokens * case["heads"] * case["hd"] * e + given,
                "flops": 12 * tokens * case["heads"] * case["n"] * case["axes"]}
    C = case["C"]
    if case["op"] == "norm":
        return {"bytes": 4 * tokens * C * e, "flops": 16 * tokens * C}
    return {"bytes": 6 * tokens * C * e, "flops": 40 * tokens * C}
