"""The norm of queries and keys with the rotation, attention and their gradients from the
definitions in 64 bits, with element-wise bounds on what bf16 storage and fp32 arithmetic may
move (test helper).

A stored bf16 value is off by at most U = 2^-8 of itself, an fp32 one by 2^-24.  With hats
for what the kernel computes:

  P^  = P (1 + e), e <= ln 2 (error of the exponent, in log2 units) + 2^-21:
        the score's fp32 sum of 128 products 2^-17 sum |q k| c, the log-sum-exp (given in
        fp32, scaled and added in fp32) 2^-22 (|lse| c'), the exponential instruction 2^-22,
        which gives zero below 2^-126; in a product, P^ is rounded to bf16: U more
  D^  : O is given in bf16 and summed in fp32: |D^ - D| <= (U + 2^-17) sum |dO| |O|, where
        O itself may be off by dO_of (what the forward pass left)
  dS^ = P^ (dP^ - D^): |dS^ - dS| <= e |dS| + P (|D^ - D| + 2^-17 sum |dO| |v|), then U |dS^|
and every sum adds 2^-17 of the sum of magnitudes (more than fp32 loses: 2^-24 a step, over
blocks that are summed apart), every output U of itself."""
import math

import torch

U = 2.0 ** -8
F = 2.0 ** -17


def heads(x, H):
    """[L][n * H * 128] -> n tensors [H][L][128] in fp64."""
    v = x.double().view(x.shape[0], -1, H, 128)
    return [v[:, i].transpose(0, 1) for i in range(v.shape[1])]


def hidden(L, cu, causal, dev):
    i = torch.arange(L, device=dev)
    hide = torch.zeros(L, L, dtype=torch.bool, device=dev)
    if cu is not None:
        seg = torch.bucketize(i, torch.tensor(list(cu[1:]), device=dev), right=True)
        hide |= seg[None] != seg[:, None]
    if causal:
        hide |= i[None] > i[:, None]
    return hide


def attention(qkv, H, causal=False, cu=None, scale=1 / math.sqrt(128)):
    """O [L][H*128] and lse [H][L], fp64."""
    L = qkv.shape[0]
    q, k, v = heads(qkv, H)
    s = (q @ k.transpose(1, 2)) * scale
    s = s.masked_fill(hidden(L, cu, causal, qkv.device), -math.inf)
    lse = torch.logsumexp(s, 2)
    O = torch.exp(s - lse[:, :, None]) @ v
    return O.transpose(0, 1).reshape(L, H * 128), lse


def attention_bwd(qkv, dO, H, causal=False, cu=None, scale=1 / math.sqrt(128), dO_of=None):
    """The exact dqkv [L][3*H*128] and the bound on each element; dO_of: how far the given O may
    be from the exact one beyond its own rounding ([L][H*128])."""
    L = qkv.shape[0]
    q, k, v = heads(qkv, H)
    (g,) = heads(dO, H)
    O, lse = attention(qkv, H, causal, cu, scale)
    (o,) = heads(O, H)
    hide = hidden(L, cu, causal, qkv.device)
    p = torch.exp((q @ k.transpose(1, 2)) * scale - lse[:, :, None]).masked_fill(hide, 0.0)
    dp = g @ v.transpose(1, 2)
    D = (p * dp).sum(2, keepdim=True)
    ds = p * (dp - D)
    out = [scale * ds @ k, scale * ds.transpose(1, 2) @ q, p.transpose(1, 2) @ g]
    e = scale * F * (q.abs() @ k.abs().transpose(1, 2)) + 2.0 ** -22 * lse.abs()[:, :, None] + 2.0 ** -21
    off_o = torch.zeros_like(o) if dO_of is None else heads(dO_of, H)[0]
    off_D = (g.abs() * ((U + F) * o.abs() + (1 + U) * off_o)).sum(2, keepdim=True)
    off_ds = e * ds.abs() + (1 + e) * p * (off_D + F * (g.abs() @ v.abs().transpose(1, 2)))
    off_ds = off_ds + 2.0 ** -126 * (dp.abs() + D.abs() + off_D)
    off_ds = off_ds + U * (ds.abs() + off_ds) + 2.0 ** -133
    off_p = p * (e + U * (1 + e)) + 2.0 ** -125
    off_ds, off_p = (x.masked_fill(hide, 0.0) for x in (off_ds, off_p))
    big_ds, big_p = ds.abs() + off_ds, p + off_p
    t = lambda x: x.transpose(1, 2)  # noqa: E731
    bound = [scale * (off_ds + F * big_ds) @ k.abs(), scale * t(off_ds + F * big_ds) @ q.abs(),
             t(off_p + F * big_p) @ g.abs()]
    # the output's own rounding; values below the normal numbers step by 2^-133
    bound = [b + U * (r.abs() + b) + 2.0 ** -133 for b, r in zip(bound, out)]
    flat = lambda xs: torch.stack(xs).permute(2, 0, 1, 3).reshape(L, -1)  # noqa: E731
    return flat(out), flat(bound)


def angles(pos, sec, base):
    """[L][64] in fp64; the call takes the base in fp32."""
    base = float(torch.tensor(base, dtype=torch.float32))
    cols = [pos[:, a].double()[:, None] * base ** (-2.0 * torch.arange(n // 2, device=pos.device).double() / n)
            for a, n in enumerate(sec)]
    return torch.cat(cols, 1)


def turn(x, ang):
    """Pairs (2j, 2j + 1) of x [L][..][128] turned by ang [L][64]."""
    while ang.dim() < x.dim():
        ang = ang[:, None]
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack((u * ang.cos() - v * ang.sin(), u * ang.sin() + v * ang.cos()), -1).flatten(-2)


def qk_norm(qkv, pos, wq, wk, H, eps, sec=(32, 48, 48), base=10000.0):
    """The exact output [L][3*H*128] and, for Q and K, the sum of magnitudes behind each
    element (for the fp32 part of a bound)."""
    L = qkv.shape[0]
    x = qkv.double().view(L, 3, H, 128)
    one = torch.ones(128, dtype=torch.float64, device=qkv.device)
    w = torch.stack([one if t is None else t.double() for t in (wq, wk)])[:, None]
    f = x[:, :2]
    r = (f.square().mean(3, keepdim=True) + eps).rsqrt()
    r = torch.where(torch.isinf(r), torch.zeros_like(r), r)
    n = f * r * w
    ang = angles(pos, sec, base)
    y = turn(n, ang)
    pair = n.view(L, 2, H, 64, 2).abs().sum(4, keepdim=True).expand(-1, -1, -1, -1, 2).reshape(n.shape)
    return (torch.cat((y, x[:, 2:]), 1).view(L, -1),
            torch.cat((pair, torch.zeros_like(x[:, 2:])), 1).view(L, -1))


def qk_norm_bwd(qkv, pos, wq, wk, dout, H, eps, sec=(32, 48, 48), base=10000.0):
    """Exact dqkv, dwq, dwk, and the sums of magnitudes behind each."""
    L = qkv.shape[0]
    x, dy = (t.double().view(L, 3, H, 128) for t in (qkv, dout))
    one = torch.ones(128, dtype=torch.float64, device=qkv.device)
    w = torch.stack([one if t is None else t.double() for t in (wq, wk)])[:, None]
    f = x[:, :2]
    r = (f.square().mean(3, keepdim=True) + eps).rsqrt()
    r = torch.where(torch.isinf(r), torch.zeros_like(r), r)
    n = f * r
    g = turn(dy[:, :2], -angles(pos, sec, base))
    big = dy[:, :2].reshape(L, 2, H, 64, 2).abs().sum(4, keepdim=True).expand(-1, -1, -1, -1, 2).reshape(g.shape)
    dw, dw_big = (g * n).sum((0, 2)), (big * n.abs()).sum((0, 2))
    gw = g * w
    dx = r * (gw - n * (gw * n).mean(3, keepdim=True))
    bigw = big * w.abs()
    dx_big = r * (bigw + n.abs() * (bigw * n.abs()).mean(3, keepdim=True))
    full = lambda a, b: torch.cat((a, b), 1).view(L, -1)  # noqa: E731
    return (full(dx, dy[:, 2:]), dw[0], dw[1]), (full(dx_big, torch.zeros_like(dy[:, 2:])), dw_big[0], dw_big[1])


def assert_within(got, ref, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got - ref).abs()
    over = off / bound.clamp(min=1e-300)
    worst = float(over.max())
    at = int(over.argmax())
    assert worst <= 1.0, (f"{what}: element {at} is {worst:.3f} of its bound: "
                          f"{float(got.flatten()[at])!r} for {float(ref.flatten()[at])!r}")
    return worst
