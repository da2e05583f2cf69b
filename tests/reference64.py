"""Plain 64-bit forms of the differential block's operators, from their definitions, with bounds on the
rounding errors of a computation that follows them in fp32 with bf16 or fp32 inputs and outputs.

Half a step of rounding is U = torch.finfo(t).eps / 2 of the value. Bounds count:
* one rounding of each output: U_out |value|;
* bf16 maps only, the rounding of P, P1 - lam P2 and dS to bf16 where they enter a product: 2^-8 of each
  term's magnitude (the CUDA-core kernels round none of them, and stay below);
* the fp32 arithmetic before it. A score of d products, added in any order, is off by at most
  (d + 2) 2^-24 mag, mag = scale sum_c |q_c k_c|; an error e of a score changes P by a factor e^(2 e) at
  most (numerator and normaliser); exp2's own relative error is at most 2^-21 (argument reduction by
  the maximum included: |score log2 e| 2^-24, counted with mag); sums of n terms add n 2^-24. So each P
  carries at most c = 2 (d + 6) 2^-24 mag + 2^-20 + 2 (n + 8) 2^-24, and a product of P with values x is
  off by c sum P |x| plus (n + 8) 2^-24 sum P |x|, which c counts already.
"""
import math

import numpy as np
import torch

F64 = torch.float64


def region_tokens(H, W, n_win):
    """List over regions of the flat token numbers, row by row."""
    hr, wr = H // n_win, W // n_win
    return [torch.tensor([(ry * hr + y) * W + rx * wr + x for y in range(hr) for x in range(wr)])
            for ry in range(n_win) for rx in range(n_win)]


def diff(q, k, v, idx, lam, heads, n_win, dout=None, low=None):
    """Forward (and, with dout, backward) in 64 bits on the CPU. low: the kernels' rounding of P and dS
    (2^-8 for bf16 maps, 0 for fp32 ones). Returns a dict of results and of their bounds ("out_tol", ...),
    without the rounding of the outputs themselves."""
    B, H, W, C = q.shape
    low = (2.0 ** -8 if q.dtype == torch.bfloat16 else 0.0) if low is None else low
    hd = C // heads
    d, N = hd // 2, H * W
    scale = 1 / math.sqrt(d)
    q, k, v = (t.detach().cpu().to(F64).view(B, N, heads, hd) for t in (q, k, v))
    lam = lam.detach().cpu().to(F64)
    idx = idx.cpu()
    toks = region_tokens(H, W, n_win)
    R = n_win * n_win
    z = lambda: torch.zeros(B, N, heads, hd, dtype=F64)
    res = {"out": z(), "out_tol": z()}
    if dout is not None:
        do = dout.detach().cpu().to(F64).view(B, N, heads, hd)
        for name in ("dq", "dk", "dv"):
            res[name], res[name + "_tol"] = z(), z()
        res["dlam"], res["dlam_tol"] = torch.zeros(heads, dtype=F64), torch.zeros(heads, dtype=F64)
    for b in range(B):
        for r in range(R):
            regions = [int(s) for s in idx[b, r] if 0 <= int(s) < R]
            if not regions:
                continue
            t, src = toks[r], torch.cat([toks[s] for s in regions])
            n = len(src)
            for h in range(heads):
                qq, kk, vv = q[b, t, h], k[b, src, h], v[b, src, h]
                lm = float(lam[h])
                halves = (slice(0, d), slice(d, hd))
                p = [torch.softmax(qq[:, i] @ kk[:, i].T * scale, -1) for i in halves]
                mag = max(float((qq[:, i].abs() @ kk[:, i].abs().T).max()) * scale for i in halves)
                c = 2 * (d + 6) * 2.0 ** -24 * mag + 2.0 ** -20 + 2 * (n + 8) * 2.0 ** -24
                both = p[0] + abs(lm) * p[1]
                res["out"][b, t, h] = (p[0] - lm * p[1]) @ vv
                res["out_tol"][b, t, h] = (low + c) * (both @ vv.abs())
                if dout is None:
                    continue
                g = do[b, t, h]
                dp = g @ vv.T
                m = g.abs() @ vv.abs().T  # what bounds dP's own error
                res["dv"][b].index_put_((src, torch.tensor(h)), (p[0] - lm * p[1]).T @ g, accumulate=True)
                nq = len(t) * R  # queries that may meet one key
                res["dv_tol"][b].index_put_((src, torch.tensor(h)), (low + c + nq * 2.0 ** -24) * (both.T @ g.abs()),
                                            accumulate=True)
                for i, w in ((0, 1.0), (1, -lm)):
                    D = (p[i] * dp).sum(-1, keepdim=True)
                    Dm = (p[i] * m).sum(-1, keepdim=True)
                    ds = p[i] * (dp - D)
                    # rounding of dS, and c of everything that went into it
                    err = p[i] * (low * (dp - D).abs() + 2 * (c + (hd + 4) * 2.0 ** -24) * (m + Dm))
                    res["dq"][b, t, h, halves[i]] += w * scale * ds @ kk[:, halves[i]]
                    res["dq_tol"][b, t, h, halves[i]] += abs(w) * scale * err @ kk[:, halves[i]].abs()
                    res["dk"][b, :, h, halves[i]].index_put_((src,), w * scale * ds.T @ qq[:, halves[i]], accumulate=True)
                    res["dk_tol"][b, :, h, halves[i]].index_put_(
                        (src,), abs(w) * scale * (err + nq * 2.0 ** -24 * ds.abs()).T @ qq[:, halves[i]].abs(),
                        accumulate=True)
                    if i == 1:
                        res["dlam"][h] -= D.sum()
                        res["dlam_tol"][h] += 2 * (c + (hd + 4) * 2.0 ** -24) * Dm.sum()
    return {name: x if name.startswith("dlam") else x.view(B, H, W, C) for name, x in res.items()}


def check(got, ref, tol, what):
    """|got - ref| <= tol + half a rounding step of got's type, element by element, and all finite."""
    u = torch.finfo(got.dtype).eps / 2
    got, ref, tol = got.detach().cpu().to(F64), ref.to(F64), tol.to(F64)
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)} against {tuple(ref.shape)}"
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    # a value that rounds lies within (1 + u) of the unrounded one, which itself is off by tol; 1e-38: the
    # smallest normal number, below which both types' steps stop shrinking
    over = (got - ref).abs() - (tol * (1 + u) + u * ref.abs() + 1e-38)
    assert float(over.max()) <= 0, (f"{what}: off by up to {float((got - ref).abs().max()):.3e}, "
                                    f"{float(over.max()):.3e} beyond its bound, at {np.unravel_index(int(over.argmax()), over.shape)}")


def rope(x, freqs, heads, layout, axes, origin, pos, mscale, inverse):
    """Rotary positions as products of complex numbers; x on the CPU."""
    B, H, W, C = x.shape
    hd, n = C // heads, freqs.numel()
    f = freqs.cpu().to(F64)
    if pos is None:
        y = torch.arange(H, dtype=F64).view(H, 1) + origin[0]
        xx = torch.arange(W, dtype=F64).view(1, W) + origin[1]
        at = torch.stack((y.expand(H, W), xx.expand(H, W)), -1) if axes == 2 else (y * W + xx).unsqueeze(-1)
        at = at.unsqueeze(0)
    else:
        at = pos.cpu().to(F64)
    ang = at[:, :, :, None, :, None] * f
    turn = torch.polar(torch.full_like(ang, mscale), -ang if inverse else ang)
    full = x.cpu().to(F64).view(B, H, W, heads, hd).clone()
    mag = full.abs()
    for a in range(axes):
        c0 = 2 * n * a
        one, two = ((slice(c0, c0 + n), slice(c0 + n, c0 + 2 * n)) if layout == "half" else
                    (slice(c0, c0 + 2 * n, 2), slice(c0 + 1, c0 + 2 * n, 2)))
        w = torch.complex(full[..., one], full[..., two])
        m = w.abs() * abs(mscale)
        w = w * turn[..., a, :]
        full[..., one], full[..., two] = w.real, w.imag
        mag[..., one], mag[..., two] = m, m
    # fp32: the angle in half turns is rounded once (2^-25 of at most one: pi 2^-25 of an angle), sine and
    # cosine are within 2^-23 each, their scaling and the two products and the sum round once each
    # (2^-24): below 2^-21 of the pair's length in all; untouched channels are copied
    tol = mag * 2.0 ** -21
    tol[..., 2 * n * axes:] = 0
    return full.view(B, H, W, C), tol.view(B, H, W, C)


def norm_residual(x, h, gate, w_post, b_post, w_pre, b_pre, alpha, eps, kind, dy=None, ds=None):
    """s, y and, with dy or ds, the gradients (automatic differentiation in 64 bits) as a dict."""
    leaf = lambda t: None if t is None else t.detach().cpu().to(F64).requires_grad_(dy is not None or ds is not None)
    names = ("x", "h", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")
    leaves = dict(zip(names, map(leaf, (x, h, gate, w_post, b_post, w_pre, b_pre))))
    x, h, gate, w_post, b_post, w_pre, b_pre = leaves.values()

    def norm(t):
        if kind == "layer":
            return (t - t.mean(-1, keepdim=True)) / torch.sqrt(t.var(-1, unbiased=False, keepdim=True) + eps)
        return t / torch.sqrt(t.square().mean(-1, keepdim=True) + eps)

    s = alpha * x
    if h is not None:
        p = h if w_post is None else norm(h) * w_post
        if b_post is not None:
            p = p + b_post
        if gate is not None:
            p = p * (gate if gate.dim() == 1 else gate[:, None, None, :])
        s = s + p
    y = None
    if w_pre is not None:
        y = norm(s) * w_pre
        if b_pre is not None:
            y = y + b_pre
    out = {"s": s.detach(), "y": None if y is None else y.detach()}
    if dy is not None or ds is not None:
        loss = sum((t * g.detach().cpu().to(F64)).sum() for t, g in ((s, ds), (y, dy)) if g is not None)
        loss.backward()
        out.update({"d" + m: None if t is None else t.grad for m, t in leaves.items()})
    return out
