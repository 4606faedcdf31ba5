"""The norm of queries and keys and the gradients on a machine without a GPU: the library
exports what include/h3attn_train.h declares and refuses bad arguments before any launch."""
import ctypes
import os
import re

import pytest
import torch

from tests import _train as tr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, WS = 1, 2, 6
P = 1 << 30          # an aligned fake address: never dereferenced on these paths
FAR = 1 << 36        # arrays this far apart do not overlap


@pytest.fixture(scope="module")
def lib():
    from joint_audio_video_gb300 import build
    build.build()
    import joint_audio_video_gb300 as h3
    return h3


def at(i):
    return P + i * FAR


def test_library_exports_every_declared_entry_point(lib):
    with open(os.path.join(ROOT, "include", "h3attn_train.h")) as f:
        names = sorted(set(re.findall(r"^\s*h3_status\s+(h3_\w+)\s*\(", f.read(), re.M)))
    assert sorted(lib.TRAIN_SYMBOLS) == names and len(names) == 6
    raw = ctypes.CDLL(lib.lib_path)
    for n in names:
        assert hasattr(raw, n) and n in lib.__all__


def test_workspace_sizes(lib):
    r = lambda n: (n + 255) // 256 * 256  # noqa: E731
    for L, H in ((1, 1), (128, 3), (129, 3), (58758, 40)):
        assert lib.h3_attn_bwd_workspace_size(L, H) == 256 + r(H * ((L + 127) // 128 * 128 + 128) * 8)
    assert lib.h3_qk_norm_mrope_bwd_workspace_size(58758, 40) == 1 << 20
    L, n = lib.load(), ctypes.c_size_t(0)
    for fn in (L.h3_attn_bwd_workspace_size, L.h3_qk_norm_mrope_bwd_workspace_size):
        for bad in ((0, 1, 128), (-1, 1, 128), (8, 0, 128), (8, 129, 128), (8, 2 ** 31 - 1, 128)):
            assert fn(*bad, ctypes.byref(n)) == INV, bad
        assert fn(8, 2, 64, ctypes.byref(n)) == UNS
        assert fn(8, 2, 128, None) == INV
    # tokens and CTAs past 31 bits
    for bad in ((2 ** 31 - 1, 1), (2 ** 30 + 1, 1), (2 ** 30, 128)):
        assert L.h3_attn_bwd_workspace_size(*bad, 128, ctypes.byref(n)) == INV, bad
    assert L.h3_attn_bwd_workspace_size(2 ** 30, 1, 128, ctypes.byref(n)) == 0
    assert n.value == 256 + (2 ** 30 + 128) * 8


def _sec(*v):
    a = (ctypes.c_int32 * 3)(*v)
    return ctypes.addressof(a), a


def test_norm_refusals(lib):
    L = lib.load()
    good, keep = _sec(32, 48, 48)
    odd, keep1 = _sec(33, 47, 48)
    short, keep2 = _sec(32, 48, 32)
    neg, keep3 = _sec(-2, 82, 48)
    need = lib.h3_qk_norm_mrope_bwd_workspace_size(64, 2)

    def fwd(qkv=at(0), pos=at(1), wq=at(2), wk=at(3), n=64, H=2, dh=128, sec=good, base=1e4, eps=1e-6,
            out=at(4)):
        return L.h3_qk_norm_mrope(qkv, pos, wq, wk, n, H, dh, sec, base, eps, out, None)

    def bwd(qkv=at(0), pos=at(1), wq=at(2), wk=at(3), dout=at(5), n=64, H=2, dh=128, sec=good, base=1e4,
            eps=1e-6, ws=at(6), nbytes=need, out=at(4), dwq=at(7), dwk=at(8)):
        return L.h3_qk_norm_mrope_bwd(qkv, pos, wq, wk, dout, n, H, dh, sec, base, eps, ws, nbytes, out,
                                      dwq, dwk, None)
    nan, inf = float("nan"), float("inf")
    for call in (fwd, bwd):
        for bad in (dict(n=0), dict(n=-4), dict(H=0), dict(H=129), dict(sec=None), dict(sec=odd),
                    dict(sec=short), dict(sec=neg), dict(base=0.0), dict(base=-2.0), dict(base=nan),
                    dict(base=inf), dict(eps=-1e-6), dict(eps=nan), dict(eps=inf), dict(qkv=None),
                    dict(pos=None), dict(out=None), dict(qkv=at(0) + 8), dict(pos=at(1) + 2),
                    dict(wq=at(2) + 4), dict(wk=at(3) + 8), dict(out=at(4) + 2), dict(out=at(0) + 16),
                    dict(out=at(1)), dict(out=at(2)), dict(out=at(3))):
            assert call(**bad) == INV, (call.__name__, bad)
        assert call(dh=64) == UNS
    for bad in (dict(dout=None), dict(dout=at(5) + 4), dict(ws=None), dict(ws=at(6) + 16), dict(out=at(0)),
                dict(out=at(5) + 16), dict(out=at(6)), dict(out=at(7)), dict(dwq=at(7) + 2),
                dict(dwk=at(8) + 1), dict(dwq=at(8)), dict(dwq=at(0)), dict(dwk=at(5)), dict(dwk=at(2)),
                dict(ws=at(0)), dict(ws=at(5)), dict(ws=at(7)), dict(ws=at(1))):
        assert bwd(**bad) == INV, bad
    assert bwd(nbytes=need - 1) == WS


def test_attention_gradient_refusals(lib):
    L = lib.load()
    need = lib.h3_attn_bwd_workspace_size(45, 2)
    size = 45 * 2 * 128 * 2

    def whole(qkv=at(0), O=at(1), lse=at(2), dO=at(3), n=45, H=2, dh=128, causal=0, scale=0.1, ws=at(4),
              nbytes=need, out=at(5)):
        return L.h3_joint_attn_bwd(qkv, O, lse, dO, n, H, dh, causal, scale, ws, nbytes, out, None)

    def parts(cu=(0, 10, 45), n_seg=None, qkv=at(0), O=at(1), lse=at(2), dO=at(3), n=45, H=2, dh=128,
              causal=0, scale=0.1, ws=at(4), nbytes=need, out=at(5)):
        a = None if cu is None else (ctypes.c_int32 * len(cu))(*cu)
        return L.h3_joint_attn_varlen_bwd(qkv, O, lse, dO, None if a is None else ctypes.addressof(a),
                                          (0 if cu is None else len(cu) - 1) if n_seg is None else n_seg, n,
                                          H, dh, causal, scale, ws, nbytes, out, None)
    for call in (whole, parts):
        for bad in (dict(n=0), dict(H=0), dict(H=200), dict(causal=2), dict(causal=-1), dict(scale=0.0),
                    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(qkv=None),
                    dict(O=None), dict(lse=None), dict(dO=None), dict(ws=None), dict(out=None),
                    dict(qkv=at(0) + 2), dict(O=at(1) + 8), dict(lse=at(2) + 2), dict(dO=at(3) + 4),
                    dict(ws=at(4) + 128), dict(out=at(5) + 8), dict(out=at(0)), dict(out=at(1)),
                    dict(out=at(2)), dict(out=at(3)), dict(out=at(4)), dict(out=at(3) - 2 * size),
                    dict(ws=at(0)), dict(ws=at(1)), dict(ws=at(2)), dict(ws=at(3))):
            assert call(**bad) == INV, (call.__name__, bad)
        assert call(dh=64) == UNS
        assert call(nbytes=need - 1) == WS
    for bad in (dict(cu=(1, 10, 45)), dict(cu=(0, 30, 10, 45)), dict(cu=(0, 44)), dict(cu=None, n_seg=1),
                dict(n_seg=0), dict(n_seg=-1), dict(cu=(0,) * 65 + (45,))):
        assert parts(**bad) == INV, bad


# ------------------------------------------------------------------ the definitions themselves
@pytest.mark.parametrize("causal,cu", [(False, None), (True, None), (False, [0, 3, 3, 9]),
                                       (True, [0, 4, 9])])
def test_gradient_formula_against_differences(causal, cu):
    """The definition's dqkv against central differences of sum(dO * O), in 64 bits."""
    g = torch.Generator().manual_seed(2)
    L, H = 9, 2
    qkv = torch.randn(L, 3 * H * 128, generator=g, dtype=torch.float64)
    dO = torch.randn(L, H * 128, generator=g, dtype=torch.float64)
    d, bound = tr.attention_bwd(qkv, dO, H, causal, cu)
    f = lambda x: float((tr.attention(x, H, causal, cu)[0] * dO).sum())  # noqa: E731
    for _ in range(6):
        u = torch.randn(qkv.shape, generator=g, dtype=torch.float64)
        diff = (f(qkv + 1e-5 * u) - f(qkv - 1e-5 * u)) / 2e-5
        assert abs(diff - float((d * u).sum())) <= 1e-7 * (1 + abs(diff))
    assert (bound > 0).all() and float((bound / d.abs().mean()).max()) < 1.0


def test_bounds_take_the_roundings_and_refuse_a_mistake():
    """bf16 roundings of P, dS and the results stay within the bounds; a lost diagonal, an
    unscaled dK or D without its last block do not."""
    g = torch.Generator().manual_seed(3)
    L, H = 70, 1
    qkv = torch.randn(L, 384, generator=g).to(torch.bfloat16).double()
    dO = torch.randn(L, 128, generator=g).to(torch.bfloat16).double()
    d, bound = tr.attention_bwd(qkv, dO, H, True)
    q, k, v = (t[0] for t in tr.heads(qkv, 1))
    s = 128 ** -0.5
    r = lambda x: x.float().to(torch.bfloat16).double()  # noqa: E731

    def emulate(diag=True, sk=s, cut=128):
        hide = torch.ones(L, L, dtype=torch.bool).triu(1 if diag else 0)
        hide[0, 0] = False
        O, lse = tr.attention(qkv, 1, True)
        p = torch.exp((q @ k.T) * s - lse[0][:, None]).masked_fill(hide, 0.0)
        ds = p * (dO @ v.T - (dO * r(O))[:, :cut].sum(1, keepdim=True))
        return torch.cat((r(s * r(ds) @ k), r(sk * r(ds).T @ q), r(r(p).T @ dO)), 1)
    assert ((emulate() - d).abs() <= bound).all()
    for wrong in (dict(diag=False), dict(sk=1.01 * s), dict(cut=120)):
        assert not ((emulate(**wrong) - d).abs() <= bound).all(), wrong


@pytest.mark.parametrize("eps", [1e-6, 0.3])
def test_norm_gradient_formula_against_autograd(eps):
    """The definition's dqkv, dwq and dwk against automatic differentiation in 64 bits, and the
    rotation's own properties: lengths kept, position 0 unturned."""
    g = torch.Generator().manual_seed(4)
    L, H, sec, base = 11, 3, (20, 60, 48), 500.0
    qkv = torch.randn(L, 3 * H * 128, generator=g, dtype=torch.float64)
    dout = torch.randn(L, 3 * H * 128, generator=g, dtype=torch.float64)
    pos = torch.randint(-40, 90, (L, 3), generator=g, dtype=torch.int32)
    pos[0] = 0
    wq, wk = (1 + 0.3 * torch.randn(128, generator=g, dtype=torch.float64) for _ in range(2))
    x, a, b = (t.clone().requires_grad_(True) for t in (qkv, wq, wk))
    y, _ = tr.qk_norm(x, pos, a, b, H, eps, sec, base)
    (y * dout).sum().backward()
    (dx, da, db), bigs = tr.qk_norm_bwd(qkv, pos, wq, wk, dout, H, eps, sec, base)
    for got, ref in ((x.grad, dx), (a.grad, da), (b.grad, db)):
        assert float((got - ref).abs().max()) <= 1e-10
    assert all((r.abs() <= m + 1e-12).all() for r, m in zip((dx[:, :2 * H * 128], da, db),
                                                           (bigs[0][:, :2 * H * 128], bigs[1], bigs[2])))
    f = qkv.view(L, 3, H, 128)[:, :2]
    n = f / (f.square().mean(3, keepdim=True) + eps).sqrt() * torch.stack((wq, wk))[:, None]
    y = y.detach().view(L, 3, H, 128)[:, :2]
    assert torch.allclose(y[0], n[0], atol=1e-12)
    assert torch.allclose(y.square().sum(3), n.square().sum(3), atol=1e-9)
