"""The 64-bit definitions themselves, on the CPU: the differential attention's gradient formulas against central
differences, its special cases against plain softmax attention, and the frequency helper."""
import math

import pytest
import torch

import bi_level_routing_b200 as bra
import reference64 as ref


def _case(B=1, hr=2, wr=3, n_win=2, topk=3, heads=2, hd=8, seed=0):
    g = torch.Generator().manual_seed(seed)
    H, W, C, R = hr * n_win, wr * n_win, heads * hd, n_win * n_win
    q, k, v, dout = (torch.randn((B, H, W, C), generator=g, dtype=ref.F64) for _ in range(4))
    idx = torch.randint(0, R, (B, R, topk), generator=g, dtype=torch.int32)
    idx[0, -1] = -1  # an empty row
    lam = torch.rand(heads, generator=g, dtype=ref.F64)
    return q, k, v, idx, lam, dout, heads, n_win


def test_gradients_against_differences():
    q, k, v, idx, lam, dout, heads, n_win = _case()
    want = ref.diff(q, k, v, idx, lam, heads, n_win, dout)
    loss = lambda *a: float((ref.diff(*a[:3], idx, a[3], heads, n_win)["out"] * dout).sum())
    g = torch.Generator().manual_seed(1)
    for i, name in enumerate(("dq", "dk", "dv", "dlam")):
        args = [q, k, v, lam]
        step = torch.randn(args[i].shape, generator=g, dtype=ref.F64)
        ends = []
        for sign in (1, -1):
            moved = list(args)
            moved[i] = args[i] + sign * 1e-5 * step
            ends.append(loss(*moved))
        slope = (ends[0] - ends[1]) / 2e-5
        # central differences: 1e-10 times third derivatives of order 10^2, and 1e-16 / 1e-5 of rounding
        assert abs(slope - float((want[name] * step).sum())) < 1e-6, name


def test_special_cases():
    q, k, v, idx, lam, _, heads, n_win = _case(n_win=1, topk=1, hr=3, wr=4)
    idx.zero_()
    lam.zero_()
    out = ref.diff(q, k, v, idx, lam, heads, n_win)["out"].view(1, 12, heads, 8)
    x = lambda t, s: t.view(1, 12, heads, 8)[..., s].transpose(1, 2)
    a = torch.nn.functional.scaled_dot_product_attention(x(q, slice(0, 4)), x(k, slice(0, 4)), x(v, slice(0, 8)))
    assert torch.allclose(out, a.transpose(1, 2), atol=1e-12)
    # equal halves and lam = 1: nothing is left
    two = lambda t: torch.cat((t.view(1, 3, 4, heads, 8)[..., :4],) * 2, -1).view(t.shape)
    assert float(ref.diff(two(q), two(k), v, idx, lam + 1, heads, n_win)["out"].abs().max()) < 1e-12


def test_rope_frequencies():
    f, m = bra.rope_frequencies(8)
    assert m == 1.0 and f.dtype == torch.float32 and float(f[0]) == 1.0
    assert torch.allclose(f, 10000.0 ** (-torch.arange(8) / 8))
    assert torch.allclose(bra.rope_frequencies(8, scaling="linear", factor=4)[0], f / 4)
    ntk = bra.rope_frequencies(8, scaling="ntk", factor=4)[0]
    assert float(ntk[0]) == 1.0 and math.isclose(float(ntk[-1]), float(f[-1]) / 4, rel_tol=1e-6)
    yarn, m = bra.rope_frequencies(64, scaling="yarn", factor=8, trained_extent=4096)
    assert math.isclose(m, 0.1 * math.log(8) + 1)
    full = bra.rope_frequencies(64)[0]
    turns = 4096 * full.double() / (2 * math.pi)
    assert torch.equal(yarn[turns > 40], full[turns > 40])
    assert torch.allclose(yarn[turns < 0.8], full[turns < 0.8] / 8)
    assert bool((yarn <= full).all()) and bool((yarn >= full / 8 * (1 - 1e-6)).all())
    for bad in (dict(n=0), dict(n=4, factor=0.5), dict(n=4, scaling="other"), dict(n=4, scaling="yarn", factor=2.0), dict(n=4, base=1.0)):
        with pytest.raises(ValueError):
            bra.rope_frequencies(**bad)


# ------------------------------------------------------------------ refusals of the C calls, before any launch

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x10000  # a 16-byte aligned non-NULL value; these calls must fail before using it


@pytest.fixture(scope="module")
def L():
    from bi_level_routing_b200 import api, build
    build.build()
    return api.lib()


def _sizes(kw):
    s = dict(B=1, H=28, W=28, C=64, heads=2, n_win=7, topk=4, dtype=1)
    s.update({m: kw.pop(m) for m in list(kw) if m in s})
    return list(s.values())


DIFF_BAD = [(dict(heads=3), INVALID), (dict(topk=50), INVALID), (dict(H=30), INVALID), (dict(dtype=2), INVALID), (dict(B=-1), INVALID),
            (dict(C=60), INVALID), (dict(heads=16), UNSUPPORTED), (dict(C=512, heads=2), UNSUPPORTED), (dict(heads=0), INVALID),
            (dict(H=33, W=33, n_win=33, topk=1), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", DIFF_BAD, ids=str)
def test_diff_rejects_sizes(L, kw, status):
    sizes = _sizes(dict(kw))
    assert L.bra_diff_attend(P, P, P, P, P, P, *sizes, None) == status
    assert L.bra_forward_diff(P, P, P, P, P, P, *sizes, None) == status
    assert L.bra_diff_attend_backward(P, P, P, P, P, P, P, P, P, P, *sizes, None) == status


def test_diff_rejects_pointers(L):
    apart = [P + (i << 24) for i in range(10)]  # buffers that share nothing
    for n, outs, fn in ((6, (5,), L.bra_diff_attend), (6, (5,), L.bra_forward_diff), (10, (6, 7, 8), L.bra_diff_attend_backward)):
        for i in range(n):
            for bad in (0, P + 2):
                p = apart[:n]
                p[i] = bad
                assert fn(*p, *_sizes({}), None) == INVALID, (fn.__name__, i, bad)
        for i in outs:  # an output over an input, or a part of it
            for j in (0, 1, 2):
                for shift in (0, 64):
                    p = apart[:n]
                    p[i] = p[j] + shift
                    assert fn(*p, *_sizes({}), None) == INVALID, (fn.__name__, i, j)
        if fn is not L.bra_diff_attend_backward:
            assert fn(*[0] * n, *_sizes(dict(B=0)), None) == OK
    # the routing limit on a region's row segment does not hold where nothing is routed
    wide = _sizes(dict(H=7, W=7 * 600, C=64, heads=1))
    assert L.bra_forward_diff(*apart[:6], *wide, None) == UNSUPPORTED
    # more (token, slot) pairs than the backward pass numbers
    many = _sizes(dict(H=1 << 12, W=1 << 12, C=8, heads=1, n_win=16, topk=256))
    far = [P + (i << 40) for i in range(10)]
    assert L.bra_diff_attend_backward(*far, *many, None) == UNSUPPORTED


def test_rope_rejects(L):
    def call(q=P, k=P + 4096 * 64, qo=P + 4096 * 128, ko=P + 4096 * 192, f=P, pos=0, y0=0, x0=0, B=1, H=8, W=8, C=64, heads=2, n=8,
             axes=2, dtype=1):
        return L.bra_rope(q, k, qo, ko, f, pos, y0, x0, B, H, W, C, heads, n, axes, 0, 0, 1.0, dtype, None)

    for kw in (dict(q=0), dict(qo=0), dict(f=0), dict(k=0), dict(ko=0), dict(q=P + 8), dict(f=P + 2), dict(pos=P + 1), dict(n=0), dict(n=9),
               dict(axes=0), dict(axes=3), dict(heads=3), dict(C=60), dict(dtype=4), dict(B=-1), dict(H=0), dict(y0=1 << 40),
               dict(qo=P + 16), dict(ko=P + 4096 * 64 + 16), dict(ko=P + 4096 * 128), dict(qo=P + 4096 * 64), dict(ko=P),
               dict(C=72, heads=8, n=1)):
        assert call(**kw) == INVALID, kw
    assert call(B=0, q=0) == OK


def test_norm_rejects(L):
    A = [P + (i << 16) for i in range(16)]

    def call(x=A[0], h=A[1], gate=A[2], gates=1, pw=A[3], pb=A[4], nw=A[5], nb=A[6], eps=1e-6, kind=0, s=A[7], y=A[8], B=2, H=4, W=4,
             C=64, dtype=1):
        return L.bra_norm_residual(x, h, gate, gates, pw, pb, nw, nb, 1.0, eps, kind, s, y, B, H, W, C, dtype, None)

    for kw in (dict(x=0), dict(s=0), dict(y=0), dict(nw=0), dict(pw=0), dict(h=0), dict(gates=0), dict(gates=3), dict(gate=0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(kind=2), dict(C=60), dict(dtype=3), dict(B=-1), dict(W=0), dict(x=A[0] + 8), dict(pw=A[3] + 4),
               dict(s=A[8]), dict(s=A[0] + 16), dict(y=A[1] + 32), dict(y=A[7] + 16),
               dict(h=0, gate=0, gates=0, pw=0, pb=0, nw=0, nb=0, y=0)):
        assert call(**kw) == INVALID, kw
    assert call(C=8200) == UNSUPPORTED
    assert call(B=0, x=0, gates=1) == OK

    def back(x=A[0], h=A[1], dy=A[2], ds=A[3], gate=A[4], gates=2, pw=A[5], pb=A[6], nw=A[7], nb=A[8], dx=A[9], dh=A[10], dg=A[11],
             dpw=A[12], dpb=A[13], dnw=A[14], dnb=A[15], B=2):
        return L.bra_norm_residual_backward(x, h, dy, ds, gate, gates, pw, pb, nw, nb, 1.0, 1e-6, 0, dx, dh, dg, dpw, dpb, dnw, dnb, B,
                                            4, 4, 64, 1, None)

    for kw in (dict(dx=0), dict(dh=0), dict(dy=0), dict(dg=0), dict(dpw=0), dict(dpb=0), dict(dnw=0), dict(dnb=0), dict(h=0), dict(pb=0),
               dict(dx=A[10]), dict(dx=A[0] + 16), dict(dh=A[2] + 16), dict(dg=A[11] + 2), dict(nw=0, nb=0, dnw=0, dnb=0, dy=0, ds=0)):
        assert back(**kw) == INVALID, kw

    # weight gradients over a weight, over each other, or a part of one
    for kw in (dict(dg=A[4]), dict(dg=A[4] + 64 * 4), dict(dpw=A[5]), dict(dpb=A[5] + 16), dict(dnw=A[8]), dict(dnb=A[14]), dict(dpw=A[11] + 256)):
        assert back(**kw) == INVALID, kw


def test_dlambda_over_lambda(L):
    apart = [P + (i << 24) for i in range(10)]
    for shift in (0, 4):  # two heads: eight bytes
        p = list(apart)
        p[9] = p[4] + shift
        assert L.bra_diff_attend_backward(*p, *_sizes({}), None) == INVALID


def test_kernels_per_call(L):
    stage1 = (64, 56, 56, 64, 1, 7, 1, 1)
    assert L.bra_kernels_per_call(b"bra_diff_attend", *stage1) == 1
    assert L.bra_kernels_per_call(b"bra_forward_diff", *stage1) == 3  # means, affinity and top-k, attention
    assert L.bra_kernels_per_call(b"bra_diff_attend_backward", *stage1) == 2  # queries, keys
    whole = (1, 64, 4096, 64, 1, 1, 1, 1)  # one region: nothing is routed, and its rows may be of any length
    assert L.bra_kernels_per_call(b"bra_forward_diff", *whole) == 1
    assert L.bra_kernels_per_call(b"bra_forward", *whole) == 0
    assert L.bra_kernels_per_call(b"bra_diff_attend", 64, 56, 56, 64, 16, 7, 1, 1) == 0  # heads of 4 channels
