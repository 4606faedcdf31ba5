"""Cases of the operators that train the attention sub-block: attention's backward
pass, which computes the probabilities again from the saved log-sum-exp, and the
norm of queries and keys of each head with the position rotation in the same pass,
forward and backward.

Each case is one pass through one operator.  With ``own`` false, ``run`` computes the
plain form in elementary torch operations in 32 bits (angles in 64); with ``own`` true
it calls the library.  ``exact`` computes the same outputs from the definitions in 64
bits.

  attn_bwd  from qkv, O, lse, dO:  P = exp(s Q K^T - lse) at the visible pairs,
            dV = P^T dO,  dS = P (dO V^T - rowsum(dO O)),  dQ = s dS K,  dK = s dS^T Q
  norm      q, k -> R (x / sqrt(mean x^2 + eps) * w) for each head's 128 values x, R the
            rotation of pair (2j, 2j + 1) of section a by pos[a] base^(-2j / n_a); v as it is
  norm_bwd  from qkv before the norm and the gradient of the norm's output: the gradient
            of qkv, and of w for queries and for keys (sums over tokens and heads)
"""
import math

import torch

own = False

DEV = "cuda"
DH = 128
EPS = 1e-6
SECTIONS = (32, 48, 48)     # head dims that follow t, h and w
BASE = 10000.0
SCALE = 1.0 / math.sqrt(DH)
# the dearest attention: a full-size request's tokens, an eighth of its heads
MOST = 58758 * 58758 * 5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest workload: latency
        {"name": "bwd_tiny", "op": "attn_bwd", "L": 64, "H": 2, "causal": False, "cu": ""},
        # the text of a request on its own: few tiles for each head
        {"name": "bwd_text", "op": "attn_bwd", "L": 358, "H": 40, "causal": False, "cu": ""},
        # the small workload
        {"name": "bwd_small", "op": "attn_bwd", "L": 4096, "H": 16, "causal": False, "cu": ""},
        # an odd number of tokens, causal
        {"name": "bwd_odd_causal", "op": "attn_bwd", "L": 4099, "H": 16, "causal": True, "cu": ""},
        # the medium workload's heads on one of eight GPUs, each modality on its own
        {"name": "bwd_segments", "op": "attn_bwd", "L": 16384, "H": 5, "causal": False, "cu": "0,384,15744,16384"},
        # the medium workload
        {"name": "bwd_medium", "op": "attn_bwd", "L": 16384, "H": 40, "causal": False, "cu": ""},
        # all tokens of a full-size request, the heads that one of eight GPUs has
        {"name": "bwd_full_split", "op": "attn_bwd", "L": 58758, "H": 5, "causal": False, "cu": ""},
        # one token's queries and keys: latency
        {"name": "norm_one_token", "op": "norm", "L": 1, "H": 40},
        # an odd number of tokens of the small workload's heads
        {"name": "norm_odd", "op": "norm", "L": 4099, "H": 16},
        # all tokens of a full-size request
        {"name": "norm_full", "op": "norm", "L": 58758, "H": 40},
        # the gradient, small workload
        {"name": "norm_bwd_small", "op": "norm_bwd", "L": 4096, "H": 16},
        # the gradient for all tokens of a full-size request
        {"name": "norm_bwd_full", "op": "norm_bwd", "L": 58758, "H": 40},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_bwd", "attn_bwd", "attn_bwd", "norm", "norm_bwd"])
    H = _log(rng, 1, 40)
    if op != "attn_bwd":
        return {"op": op, "L": _log(rng, 1, 58758), "H": H}
    L = _log(rng, 1, min(58758, math.isqrt(MOST // H)))
    cuts = sorted(rng.randint(0, L) for _ in range(rng.choice([0, 0, 1, 2, 6])))
    cu = ",".join(map(str, [0] + cuts + [L])) if cuts else ""
    return {"op": op, "L": L, "H": H, "causal": rng.random() < 0.4, "cu": cu}


def _segments(case):
    return [int(c) for c in case["cu"].split(",")] if case["cu"] else [0, case["L"]]


def work(case):
    L, H = case["L"], case["H"]
    n = L * H * DH
    if case["op"] == "attn_bwd":
        cu = _segments(case)
        pairs = sum((b - a) * (b - a + 1) // 2 if case["causal"] else (b - a) ** 2 for a, b in zip(cu, cu[1:]))
        # qkv, O, dO and lse read, dqkv written; five products
        return {"bytes": 16 * n + 4 * L * H, "flops": 10 * DH * H * pairs}
    if case["op"] == "norm":
        return {"bytes": 12 * n + 12 * L + 8 * DH, "flops": 2 * 10 * n}
    return {"bytes": 16 * n + 12 * L + 16 * DH, "flops": 2 * 20 * n}


# ------------------------------------------------------------------ what a program has in hand
def _hidden(cu, case):
    """Truth of "key j is not visible to query i" [L][L], or None."""
    L = case["L"]
    at = torch.arange(L, device=DEV)
    hide = None
    if case["causal"]:
        hide = at[None, :] > at[:, None]
    if len(cu) > 2:
        seg = torch.bucketize(at, torch.tensor(cu[1:], device=DEV), right=True)
        other = seg[None, :] != seg[:, None]
        hide = other if hide is None else hide.logical_or_(other)
    return hide


def _heads(x, H):
    """[L][3 or 1][H][128] of any layout -> [H][L][128] for each part, fp32."""
    L = x.shape[0]
    parts = x.view(L, -1, H, DH)
    return [parts[:, i].transpose(0, 1).float() for i in range(parts.shape[1])]


def _attention(case, qkv):
    """O (bf16) and the log-sum-exp of the scores (fp32), as the forward pass leaves them."""
    L, H = case["L"], case["H"]
    q, k, v = _heads(qkv, H)
    s = torch.matmul(q.mul_(SCALE), k.transpose(1, 2))
    hide = _hidden(_segments(case), case)
    if hide is not None:
        s.masked_fill_(hide, -math.inf)
    top = s.amax(2, keepdim=True)
    s.sub_(top).exp_()
    sums = s.sum(2, keepdim=True)
    O = torch.matmul(s, v).div_(sums)
    lse = (top + torch.log(sums)).squeeze(2)
    return O.transpose(0, 1).reshape(L, H * DH).to(torch.bfloat16), lse.contiguous()


def _positions(L):
    """(t, h, w) of a packed sequence: a little text, video frames of 45 x 40, audio on two channels."""
    n = torch.arange(L, device=DEV)
    text, audio = min(358, L // 8), L // 64 // 2 * 2
    video = L - text - audio
    v, a, step = n - text, n - text - video, max(1, audio // 2)
    one = torch.stack((n, n, n), 1)
    two = torch.stack((v // 1800, v // 40 % 45, v % 40), 1)
    three = torch.stack((a % step, torch.zeros_like(a), a // step), 1)
    rows = torch.where((n < text)[:, None], one, torch.where((n < text + video)[:, None], two, three))
    return rows.to(torch.int32).contiguous()


def prepare(case, seed):
    c = case
    L, H = c["L"], c["H"]
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows = lambda parts: torch.randn(L, parts * H * DH, generator=g, device=DEV)  # noqa: E731
    st = {"case": c}
    if c["op"] == "attn_bwd":
        st["qkv"] = rows(3).to(torch.bfloat16)
        # gradients are small, and of different size from token to token
        st["dO"] = (0.01 * rows(1) * torch.exp(0.5 * torch.randn(L, 1, generator=g, device=DEV))).to(torch.bfloat16)
        st["O"], st["lse"] = _attention(c, st["qkv"])
        st["cu"] = _segments(c) if c["cu"] else None
        st["dqkv"] = torch.empty(L, 3 * H * DH, dtype=torch.bfloat16, device=DEV)
        # the workspace that a program keeps: log-sum-exp and row sums, and room for a split of few rows
        st["room"] = torch.empty(8 * H * (L + 256) + (64 << 20), dtype=torch.uint8, device=DEV)
        return st
    # projections before the norm: tokens of different size
    st["qkv"] = (rows(3) * torch.exp(0.5 * torch.randn(L, 1, generator=g, device=DEV))).to(torch.bfloat16)
    st["wq"] = 1.0 + 0.2 * torch.randn(DH, generator=g, device=DEV)
    st["wk"] = 1.0 + 0.2 * torch.randn(DH, generator=g, device=DEV)
    st["pos"] = _positions(L)
    st["out"] = torch.empty_like(st["qkv"])
    if c["op"] == "norm_bwd":
        st["dout"] = (0.01 * rows(3)).to(torch.bfloat16)
        st["dwq"], st["dwk"] = (torch.empty(DH, device=DEV) for _ in range(2))
        st["room"] = torch.empty(2 << 20, dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------ one pass
def _run_own(st):
    import joint_audio_video_gb300 as h3
    c = st["case"]
    L, H = c["L"], c["H"]
    if c["op"] == "attn_bwd":
        room = st["room"]
        if st["cu"] is None:
            h3.h3_joint_attn_bwd(st["qkv"], st["O"], st["lse"], st["dO"], L, H, DH, c["causal"], SCALE,
                                 room, room.numel(), st["dqkv"])
        else:
            h3.h3_joint_attn_varlen_bwd(st["qkv"], st["O"], st["lse"], st["dO"], st["cu"], L, H, DH, c["causal"],
                                        SCALE, room, room.numel(), st["dqkv"])
        return _named(st["dqkv"], H)
    if c["op"] == "norm":
        h3.h3_qk_norm_mrope(st["qkv"], st["pos"], st["wq"], st["wk"], L, H, DH, EPS, st["out"], SECTIONS, BASE)
        return st["out"]
    h3.h3_qk_norm_mrope_bwd(st["qkv"], st["pos"], st["wq"], st["wk"], st["dout"], L, H, DH, EPS, st["room"],
                            st["room"].numel(), st["out"], st["dwq"], st["dwk"], SECTIONS, BASE)
    return {**_named(st["out"], H), "dwq": st["dwq"], "dwk": st["dwk"]}


def _named(dqkv, H):
    d = H * DH
    return {"dq": dqkv[:, :d], "dk": dqkv[:, d:2 * d], "dv": dqkv[:, 2 * d:]}


def _tables(pos):
    """cos and sin [L][64] of the rotation's angles, the angles in 64 bits."""
    freq = torch.cat([BASE ** (-2.0 * torch.arange(n // 2, dtype=torch.float64, device=DEV) / n) for n in SECTIONS])
    axis = torch.cat([torch.full((n // 2,), a, device=DEV) for a, n in enumerate(SECTIONS)])
    angle = pos.double()[:, axis] * freq
    return torch.cos(angle), torch.sin(angle)


def _turn(x, cos, sin):
    """Pairs (2j, 2j + 1) of x [L][..][128] turned by the angle of [L][64]."""
    u, v = x[..., 0::2], x[..., 1::2]
    c, s = (t[:, None, None, :] for t in (cos, sin))
    return torch.stack((u * c - v * s, u * s + v * c), dim=-1).flatten(-2)


def _of_bf16(x, L):
    return x.reshape(L, -1).to(torch.bfloat16)


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    L, H = c["L"], c["H"]
    if c["op"] == "attn_bwd":
        q, k, v = _heads(st["qkv"], H)
        (dO,), (O,) = _heads(st["dO"], H), _heads(st["O"], H)
        p = torch.matmul(q * SCALE, k.transpose(1, 2))
        p.sub_(st["lse"][:, :, None]).exp_()
        hide = _hidden(_segments(c), c)
        if hide is not None:
            p.masked_fill_(hide, 0.0)
        dv = torch.matmul(p.transpose(1, 2), dO)
        ds = torch.matmul(dO, v.transpose(1, 2))
        ds.sub_((dO * O).sum(2, keepdim=True)).mul_(p)
        dq = torch.matmul(ds, k).mul_(SCALE)
        dk = torch.matmul(ds.transpose(1, 2), q).mul_(SCALE)
        return {n: _of_bf16(x.transpose(0, 1), L) for n, x in (("dq", dq), ("dk", dk), ("dv", dv))}
    cos, sin = (t.float() for t in _tables(st["pos"]))
    x = st["qkv"].view(L, 3, H, DH)
    f = x[:, :2].float()
    w = torch.stack((st["wq"], st["wk"]))[None, :, None, :]
    inv = torch.rsqrt(f.square().mean(3, keepdim=True) + EPS)
    n = f * inv
    if c["op"] == "norm":
        y = _turn(n * w, cos, sin).to(torch.bfloat16)
        return torch.cat((y, x[:, 2:]), 1).view(L, 3 * H * DH)
    dout = st["dout"].view(L, 3, H, DH)
    g = _turn(dout[:, :2].float(), cos, -sin)
    dw = (g * n).sum((0, 2))
    g = g * w
    d = (inv * (g - n * (g * n).mean(3, keepdim=True))).to(torch.bfloat16)
    return {"dq": d[:, 0].reshape(L, -1), "dk": d[:, 1].reshape(L, -1), "dv": dout[:, 2].reshape(L, -1),
            "dwq": dw[0], "dwk": dw[1]}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_attention(case, st):
    """The gradient of softmax attention from q, k, v and dO alone, a head and a segment at a time."""
    L, H = case["L"], case["H"]
    qkv, dO = st["qkv"].double().view(L, 3, H, DH), st["dO"].double().view(L, H, DH)
    out = torch.zeros(3, L, H, DH, dtype=torch.float64, device=DEV)
    cu = _segments(case)
    for a, b in zip(cu, cu[1:]):
        for h in range(H if b > a else 0):
            q, k, v = (qkv[a:b, i, h] for i in range(3))
            s = (q @ k.T) / math.sqrt(DH)
            if case["causal"]:
                s = torch.where(torch.ones_like(s, dtype=torch.bool).tril(), s, torch.full_like(s, -math.inf))
            p = torch.softmax(s, dim=1)
            dp = dO[a:b, h] @ v.T
            ds = p * (dp - (p * dp).sum(1, keepdim=True))
            out[0, a:b, h] = ds @ k / math.sqrt(DH)
            out[1, a:b, h] = ds.T @ q / math.sqrt(DH)
            out[2, a:b, h] = p.T @ dO[a:b, h]
    return {n: out[i].reshape(L, H * DH) for i, n in enumerate(("dq", "dk", "dv"))}


def _rotations(pos):
    """The rotation of each token as complex numbers [L][64]."""
    angle = torch.empty(pos.shape[0], DH // 2, dtype=torch.float64, device=DEV)
    at = 0
    for a, n in enumerate(SECTIONS):
        for j in range(n // 2):
            angle[:, at] = pos[:, a].double() / BASE ** (2.0 * j / n)
            at += 1
    return torch.polar(torch.ones_like(angle), angle)


def exact(case, seed):
    c = case
    L, H = c["L"], c["H"]
    if c["op"] == "attn_bwd" and 14 * DH * L * L * H > 4e12:
        return None             # minutes in 64 bits
    st = prepare(case, seed)
    if c["op"] == "attn_bwd":
        return _exact_attention(c, st)
    turn = _rotations(st["pos"])[:, None, :]
    x = st["qkv"].view(L, 3, H, DH)
    grads, outs = [], [[], []]
    for part, w in enumerate((st["wq"].double(), st["wk"].double())):
        f = x[:, part].double()
        root = torch.sqrt((f * f).mean(2, keepdim=True) + EPS)
        if c["op"] == "norm":
            y = torch.view_as_complex((f / root * w).view(L, H, DH // 2, 2)) * turn
            outs[part] = torch.view_as_real(y).reshape(L, H * DH)
            continue
        dy = st["dout"].view(L, 3, H, DH)[:, part].double().view(L, H, DH // 2, 2)
        g = torch.view_as_real(torch.view_as_complex(dy.contiguous()) * turn.conj()).reshape(L, H, DH)
        grads.append((g * f / root).sum((0, 1)))
        g = g * w
        outs[part] = (g / root - f * (g * f).mean(2, keepdim=True) / root ** 3).reshape(L, H * DH)
    if c["op"] == "norm":
        return torch.cat((outs[0], outs[1], x[:, 2].reshape(L, H * DH).double()), 1)
    dv = st["dout"].view(L, 3, H, DH)[:, 2].reshape(L, H * DH).double()
    return {"dq": outs[0], "dk": outs[1], "dv": dv, "dwq": grads[0], "dwk": grads[1]}
