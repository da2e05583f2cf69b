"""The differential block's C calls refuse outputs that share memory with any input, the small ones (index, weights,
gate, positions) too, or with each other: other CTAs still read what one has written over. Nothing is launched."""
import pytest

INVALID = 1
BASE, STEP = 1 << 20, 1 << 24  # buffers far apart; made-up addresses, which a refused call never reads


@pytest.fixture(scope="module")
def L():
    from bi_level_routing_b200 import api, build
    build.build()
    return api.lib()


def over(written, read, in_place=()):
    """(written, read) pairs that must not meet; pairs of maps in `in_place` may be one buffer, but not a part of it."""
    return [(w, r, (w, r) in in_place) for w in written for r in read if w != r] + \
        [(w, r, False) for i, w in enumerate(written) for r in written[:i]]


def check(call, sizes, pairs):
    """call(**addresses): every pair once as one buffer and with either end inside the other."""
    place = {name: BASE + i * STEP for i, name in enumerate(sizes)}
    for w, r, same_is_fine in pairs:
        # 16-byte steps keep every buffer aligned; the last 16 bytes of one over the first of the other, both ways
        for at in ((place[r],) if not same_is_fine else ()) + (place[r] + max(0, (sizes[r] - 1) // 16 * 16), place[r] - (sizes[w] - 1) // 16 * 16):
            if same_is_fine and at == place[r]:
                continue
            assert call(**{**place, w: at}) == INVALID, (w, r, hex(at - place[r]))


B, H, W, C, HEADS, N_WIN, TOPK = 2, 8, 8, 64, 8, 2, 3
SHAPE = (B, H, W, C, HEADS, N_WIN, TOPK, 1)
MAP, IDX, LAM, ROW = B * H * W * C * 2, B * N_WIN * N_WIN * TOPK * 4, HEADS * 4, C * 4


def test_diff_attend(L):
    sizes = dict(q=MAP, k=MAP, v=MAP, idx=IDX, lam=LAM, out=MAP)
    check(lambda q, k, v, idx, lam, out: L.bra_diff_attend(q, k, v, idx, lam, out, *SHAPE, None), sizes, over(["out"], list(sizes)))


def test_forward_diff(L):
    sizes = dict(q=MAP, k=MAP, v=MAP, idx=IDX, lam=LAM, out=MAP)
    check(lambda q, k, v, idx, lam, out: L.bra_forward_diff(q, k, v, idx, lam, out, *SHAPE, None), sizes,
          over(["out", "idx"], ["q", "k", "v", "lam"]))


def test_diff_attend_backward(L):
    sizes = dict(q=MAP, k=MAP, v=MAP, idx=IDX, lam=LAM, dout=MAP, dq=MAP, dk=MAP, dv=MAP, dlam=LAM)
    check(lambda **a: L.bra_diff_attend_backward(*(a[n] for n in sizes), *SHAPE, None), sizes,
          over(["dq", "dk", "dv", "dlam"], ["q", "k", "v", "idx", "lam", "dout"]))


@pytest.mark.parametrize("axes", [1, 2])
def test_rope(L, axes):
    n = 4
    sizes = dict(q=MAP, k=MAP, q_out=MAP, k_out=MAP, freqs=4 * n, pos=B * H * W * axes * 4)

    def call(q, k, q_out, k_out, freqs, pos):
        return L.bra_rope(q, k, q_out, k_out, freqs, pos, 0, 0, B, H, W, C, 2, n, axes, 0, 0, 1.0, 1, None)

    check(call, sizes, over(["q_out", "k_out"], ["q", "k", "freqs", "pos"], in_place=[("q_out", "q"), ("k_out", "k")]))
    only_q = {m: s for m, s in sizes.items() if m not in ("k", "k_out")}
    check(lambda **a: call(k=0, k_out=0, **a), only_q, over(["q_out"], ["freqs", "pos"]))


@pytest.mark.parametrize("gates", [1, B])
def test_norm_residual(L, gates):
    sizes = dict(x=MAP, h=MAP, gate=gates * ROW, pw=ROW, pb=ROW, nw=ROW, nb=ROW, s=MAP, y=MAP)

    def call(x, h, gate, pw, pb, nw, nb, s, y):
        return L.bra_norm_residual(x, h, gate, gates, pw, pb, nw, nb, 1.0, 1e-6, 0, s, y, B, H, W, C, 1, None)

    check(call, sizes, over(["s", "y"], ["x", "h", "gate", "pw", "pb", "nw", "nb"], in_place=[(o, i) for o in "sy" for i in "xh"]))


@pytest.mark.parametrize("gates", [1, B])
def test_norm_residual_backward(L, gates):
    maps, rows = ["x", "h", "dy", "ds"], ["gate", "pw", "pb", "nw", "nb"]
    sizes = dict(x=MAP, h=MAP, dy=MAP, ds=MAP, gate=gates * ROW, pw=ROW, pb=ROW, nw=ROW, nb=ROW, dx=MAP, dh=MAP, dgate=gates * ROW,
                 dpw=ROW, dpb=ROW, dnw=ROW, dnb=ROW)

    def call(x, h, dy, ds, gate, pw, pb, nw, nb, dx, dh, dgate, dpw, dpb, dnw, dnb):
        return L.bra_norm_residual_backward(x, h, dy, ds, gate, gates, pw, pb, nw, nb, 1.0, 1e-6, 0, dx, dh, dgate, dpw, dpb, dnw, dnb,
                                            B, H, W, C, 1, None)

    check(call, sizes, over(["dx", "dh", "dgate", "dpw", "dpb", "dnw", "dnb"], maps + rows,
                            in_place=[(o, i) for o in ("dx", "dh") for i in maps]))
