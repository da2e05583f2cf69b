"""Inputs on which dq shows how dS was rounded on its way into dS k.

A row's dS sum to 0, so a channel in which all keys are alike gets dq = 0, the sum of dS; what rounding leaves of that sum is
the rounding's own. Here dP is x for three keys of four and -3 x for the fourth, x = 1 + 7 2^-10: neither truncating both to
bf16 (1 and 3 + 2^-6) nor rounding them (1 + 2^-7 and 3 + 2^-6) keeps 3 x - 3 x = 0, each off by 2^-7 of the key's
probability or more for a group of four. Two bf16 terms (the value truncated, the rest rounded) are within 2^-15 of
each dS: the first leaves a rest below 2^-7 of the value, the second rounds it by at most 2^-8 of that.

The first map's queries are 0: all its probabilities are alike. The second map's keys have two levels of scores, in whole
groups of four, so that its dS are others than the first's."""
import torch

LEVEL = 0.7  # in a channel where the query has 1
ALIKE = 1    # the channel of each half in which all keys are 1


def inputs(hr, wr, n_win, hd, seed=0):
    """q, k, v, idx (every region), lam, dout of one image and one head, bf16 on the CPU."""
    g = torch.Generator().manual_seed(seed)
    H, W, R, d = hr * n_win, wr * n_win, n_win * n_win, hd // 2
    N = H * W
    assert N % 8 == 0
    q, v, dout = (torch.zeros((N, hd)) for _ in range(3))
    k = torch.randn((N, hd), generator=g)
    k[:, [ALIKE, d + ALIKE]] = 1.0
    q[:, d] = 1.0
    j = torch.arange(N)
    k[:, d] = torch.where((j // 4) % 2 == 0, LEVEL, -LEVEL)
    sign = torch.where(j % 4 == 3, -3.0, 1.0)
    v[:, 2], v[:, 3] = sign, sign * 7 * 2.0 ** -10
    dout[:, 2:4] = 1.0
    q, k, v, dout = (t.view(1, H, W, hd).to(torch.bfloat16) for t in (q, k, v, dout))
    return q, k, v, torch.arange(R, dtype=torch.int32).expand(1, R, R).contiguous(), torch.tensor([0.6]), dout


def truncated(x):
    """64-bit values cut to bf16's eight significant bits."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.trunc(m * 256) / 256, e)


def rounded(x):
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256) / 256, e)


def dq_of(q, k, v, lam, dout, split):
    """dq in 64 bits with dS of the two maps passed through split(dS1, dS2)."""
    shape, hd = q.shape, q.shape[-1]
    d = hd // 2
    q, k, v, do = (t.double().reshape(-1, hd) for t in (q, k, v, dout))
    halves, dp, ds = (slice(0, d), slice(d, hd)), do @ v.T, []
    for s in halves:
        p = torch.softmax(q[:, s] @ k[:, s].T / d ** 0.5, -1)
        ds.append(p * (dp - (p * dp).sum(-1, keepdim=True)))
    ds = split(*ds)
    w = (1.0, -float(lam[0]))
    return torch.cat([w[i] * d ** -0.5 * ds[i] @ k[:, halves[i]] for i in (0, 1)], -1).view(shape)
