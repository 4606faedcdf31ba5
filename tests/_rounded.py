"""Attention's gradient in 64 bits with the kernel's roundings and no others (P and dS to bf16
on their way into a product, D from the stored O, each gradient once), and a comparison in the
2-norm that sees a block of rows left out of a long sum (test helper).

Element-wise bounds add up the magnitudes of all terms, values and errors grow like the root of
their number: over 58,758 terms a bound of 2^-8 of the magnitudes is some fifty times the error,
and four blocks of 128 rows may be missing below it.  The kernel differs from the chain by fp32
arithmetic alone: a rounding now and then falls the other way (its argument is off by 2^-17,
its step is 2^-8: one in hundreds), so the errors' norms agree to percents; they are held to 1.5
times the chain's, and fp32's own share to 2^-10 of the result's norm (at most 3,680 steps of 16
terms, each off by 2^-23 of the running sum: 2^-11).  A block of 128 rows out of n changes a
result by sqrt(128 / n): 5 % of it for 58,758, where the chain's error is 0.2 to 0.4 %."""
import math

import torch

from tests import _train as tr

SCALE = 1 / math.sqrt(128)


def rnd(x):
    return x.float().to(torch.bfloat16).double()


def one_head(at, q, k, v, g, lse, D, seen=None, r=lambda x: x, scale=SCALE, lost=None):
    """(dQ, dK, dV) of the tokens `at` of one head, [3][len(at)][128]; seen(i, j): truth of "query
    i sees key j" for index tensors; r: the rounding; lost: a slice of streamed tokens that the
    sums leave out (a mistake, for testing the comparison)."""
    n = torch.arange(q.shape[0], device=q.device)

    def take(p, ds):
        if lost is not None:
            p[:, lost] = 0.0
            ds[:, lost] = 0.0
        return r(p), r(ds)

    p = torch.exp((q[at] @ k.T) * scale - lse[at, None])
    if seen is not None:
        p *= seen(at[:, None], n[None])
    ds = take(p, p * (g[at] @ v.T - D[at, None]))[1]
    dq = r(scale * (ds @ k))
    p = torch.exp((k[at] @ q.T) * scale - lse[None])
    if seen is not None:
        p *= seen(n[None], at[:, None])
    p, ds = take(p, p * (v[at] @ g.T - D[None]))
    return torch.stack((dq, r(scale * (ds @ q)), r(p @ g)))


def visible(L, causal, cu, dev):
    """seen(i, j) for one_head, or None if every query sees every key."""
    if not causal and cu is None:
        return None
    seg = torch.bucketize(torch.arange(L, device=dev), torch.tensor(list((cu or [0, L])[1:]), device=dev),
                          right=True)
    return lambda i, j: ((seg[i] == seg[j]) & ((j <= i) if causal else True)).double()


def forward_one_head(q, k, v, seen=None, scale=SCALE, rows=2048):
    """O [L][128] and lse [L] in 64 bits, some rows at a time."""
    O, lse = [], []
    n = torch.arange(q.shape[0], device=q.device)
    for i in n.split(rows):
        s = (q[i] @ k.T) * scale
        if seen is not None:
            s = s.masked_fill(seen(i[:, None], n[None]) == 0, -math.inf)
        lse.append(torch.logsumexp(s, 1))
        O.append(torch.exp(s - lse[-1][:, None]) @ v)
    return torch.cat(O), torch.cat(lse)


def worst_ratio(got, exact, chain, rows=128):
    """The largest ratio of the kernel's error to what it may be, over blocks of rows of dQ, dK and
    dV apart, and where."""
    worst, where = 0.0, None
    for part, name in enumerate(("dQ", "dK", "dV")):
        g, e, c = (x[part].double().split(rows) for x in (got, exact, chain))
        share = 2.0 ** -10 * float(exact[part].norm()) / math.sqrt(len(g))
        for b, (x, y, z) in enumerate(zip(g, e, c)):
            ratio = float((x - y).norm()) / (1.5 * float((z - y).norm()) + share)
            if not ratio <= worst:
                worst, where = ratio, (name, b * rows)
    return worst, where


def check_head(got, at, head, seen, scale=SCALE, what="", rows=128, OL=None):
    """got [3][len(at)][128] against the definitions; head: (q, k, v, g) [L][128] fp64; OL: O and lse
    in 64 bits, where they are there already."""
    q, k, v, g = head
    O, lse = forward_one_head(q, k, v, seen, scale) if OL is None else OL
    exact = one_head(at, q, k, v, g, lse, (g * O).sum(1), seen, scale=scale)
    chain = one_head(at, q, k, v, g, lse, (g * rnd(O)).sum(1), seen, rnd, scale)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst, where = worst_ratio(got, exact, chain, rows)
    assert worst <= 1.0, f"{what}: {where[0]} from token {where[1]} on: {worst:.2f} of what its error may be"
    return worst


def head_of(qkv, dO, h, H):
    return tuple(t[h] for t in tr.heads(qkv, H)) + (tr.heads(dO, H)[0][h],)
