"""A training step's way through the attention sub-block: norm of queries and keys with the
rotation, attention forward, its gradient, the gradient of the norm, each call on what the
call before left, against the whole chain in 64 bits (autograd of the definitions).

Between the calls everything is stored in bf16, so the chain's error is that of a chain with the
same roundings: the test builds it in 64 bits (q, k after the norm, P, O, dS, dQ, dK, dV and
the results rounded to bf16, nothing else) and holds the kernels' error, in the 2-norm of each
result, to 1.5 times that chain's.  Both are sums of many independent roundings, so their norms
agree to a few percent; a lost term or scale moves them by far more."""
import math

import pytest
import torch

from tests import _train as tr

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1 / math.sqrt(128)
EPS = 1e-6


def rnd(x):
    return x.float().to(torch.bfloat16).double()


def exact_chain(qkv, pos, wq, wk, dO, H, causal, cu):
    x = qkv.double().requires_grad_(True)
    a, b = (w.double().requires_grad_(True) for w in (wq, wk))
    y, _ = tr.qk_norm(x, pos, a, b, H, EPS)
    O, _ = tr.attention(y, H, causal, cu)
    (O * dO.double()).sum().backward()
    return O.detach(), x.grad, a.grad, b.grad


def rounded_chain(qkv, pos, wq, wk, dO, H, causal, cu):
    L = qkv.shape[0]
    y = rnd(tr.qk_norm(qkv, pos, wq, wk, H, EPS)[0])
    q, k, v = tr.heads(y, H)
    (g,) = tr.heads(dO, H)
    s = ((q @ k.transpose(1, 2)) * SCALE).masked_fill(tr.hidden(L, cu, causal, DEV), -math.inf)
    p = torch.softmax(s, 2)
    o = rnd(rnd(p) @ v)
    ds = rnd(p * (g @ v.transpose(1, 2) - (g * o).sum(2, keepdim=True)))
    d = torch.stack([rnd(SCALE * ds @ k), rnd(SCALE * ds.transpose(1, 2) @ q), rnd(rnd(p).transpose(1, 2) @ g)])
    dy = d.permute(2, 0, 1, 3).reshape(L, -1)
    (dx, da, db), _ = tr.qk_norm_bwd(qkv, pos, wq, wk, dy, H, EPS)
    return o.transpose(0, 1).reshape(L, -1), rnd(dx), da, db


@pytest.mark.parametrize("L,H,causal,cu,in_place", [
    (64, 2, False, None, False), (333, 3, True, None, False), (1030, 2, False, None, True),
    (700, 2, False, [0, 90, 600, 700], False), (700, 2, True, [0, 90, 600, 700], True)])
def test_training_step(h3, L, H, causal, cu, in_place):
    g = torch.Generator().manual_seed(L)
    d = H * 128
    qkv = (torch.randn(L, 3 * d, generator=g) * torch.exp(0.3 * torch.randn(L, 1, generator=g))
           ).to(torch.bfloat16).to(DEV)
    pos = torch.randint(0, 50, (L, 3), generator=g, dtype=torch.int32).to(DEV)
    wq, wk = ((1.2 + 0.2 * torch.randn(128, generator=g)).to(DEV) for _ in range(2))
    dO = torch.randn(L, d, generator=g).to(torch.bfloat16).to(DEV)

    y, O = torch.empty_like(qkv), torch.empty(L, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(H, L, device=DEV)
    n1, n2 = h3.h3_attn_bwd_workspace_size(L, H), h3.h3_qk_norm_mrope_bwd_workspace_size(L, H)
    ws = torch.empty(max(n1, n2), dtype=torch.uint8, device=DEV)     # one after the other
    dy = torch.empty_like(qkv)
    dx = dy if in_place else torch.empty_like(qkv)
    dwq, dwk = torch.empty(128, device=DEV), torch.empty(128, device=DEV)

    def step():
        h3.h3_qk_norm_mrope(qkv, pos, wq, wk, L, H, 128, EPS, y)
        if cu is None:
            h3.h3_joint_attn_fwd(y, L, H, 128, causal, SCALE, O, lse)
            h3.h3_joint_attn_bwd(y, O, lse, dO, L, H, 128, causal, SCALE, ws, ws.numel(), dy)
        else:
            h3.h3_joint_attn_varlen_fwd(y, cu, L, H, 128, causal, SCALE, O, lse)
            h3.h3_joint_attn_varlen_bwd(y, O, lse, dO, cu, L, H, 128, causal, SCALE, ws, ws.numel(), dy)
        h3.h3_qk_norm_mrope_bwd(qkv, pos, wq, wk, dy, L, H, 128, EPS, ws, ws.numel(), dx, dwq, dwk)

    step()
    assert h3.h3_sync_status() == 0
    exact = exact_chain(qkv, pos, wq, wk, dO, H, causal, cu)
    same = rounded_chain(qkv, pos, wq, wk, dO, H, causal, cu)
    got = (O, dx, dwq, dwk)
    for name, a, b, c in zip(("O", "dqkv", "dwq", "dwk"), got, exact, same):
        off, fair = float((a.double() - b).norm()), float((c - b).norm())
        assert off <= 1.5 * fair, f"{name}: {off / float(b.norm()):.2e}, the rounded chain {fair / float(b.norm()):.2e}"

    # the whole step in a graph: the same bits
    first = [t.clone() for t in (y, O, lse, dx, dwq, dwk)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        step()
    for t in (y, O, lse, dx, dwq, dwk):
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert h3.h3_sync_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(first, (y, O, lse, dx, dwq, dwk)))


def test_two_steps_at_once(h3):
    """Steps on two streams, a workspace and outputs each, and a step in a graph that is replayed
    beside another on a third: the bits of a step alone."""
    L, H = 900, 3
    g = torch.Generator().manual_seed(1)
    sets = []
    for i in range(3):
        qkv = torch.randn(L, 3 * H * 128, generator=g).to(torch.bfloat16).to(DEV)
        dO = torch.randn(L, H * 128, generator=g).to(torch.bfloat16).to(DEV)
        n = h3.h3_attn_bwd_workspace_size(L, H)
        sets.append(dict(qkv=qkv, dO=dO, O=torch.empty_like(dO), lse=torch.empty(H, L, device=DEV),
                         ws=torch.empty(n, dtype=torch.uint8, device=DEV), out=torch.empty_like(qkv)))

    def step(t, stream=None):
        h3.h3_joint_attn_fwd(t["qkv"], L, H, 128, False, SCALE, t["O"], t["lse"], stream=stream)
        h3.h3_joint_attn_bwd(t["qkv"], t["O"], t["lse"], t["dO"], L, H, 128, False, SCALE, t["ws"],
                             t["ws"].numel(), t["out"], stream=stream)

    for t in sets:
        step(t)
    torch.cuda.synchronize()
    alone = [t["out"].clone() for t in sets]
    streams = [torch.cuda.Stream() for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(streams[2]), torch.cuda.graph(graph, stream=streams[2]):
        step(sets[2])
    for t in sets:
        t["out"].fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(4):
        step(sets[0], streams[0])
        step(sets[1], streams[1])
        with torch.cuda.stream(streams[2]):
            graph.replay()
    torch.cuda.synchronize()
    assert h3.h3_sync_status() == 0
    assert all(torch.equal(t["out"], a) for t, a in zip(sets, alone))
