"""The norm of each head's queries and keys with the rotation, and its gradient, against the
definitions in 64 bits: element-wise bounds from counted roundings (one to bf16; fp32
arithmetic of a few steps on the magnitudes behind each element)."""
import pytest
import torch

import joint_audio_video_gb300 as h3lib
from tests import _train as tr
from tests.test_gpu_checked import _both, checked  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"
# fp32: the mean of squares 2^-17 at most (128 terms; half of it in the root), its root, three
# products, the angle to 2^-22 and a sum of two: far below this share of the magnitudes
FWD = 2.0 ** -16
# the gradient has two such means
BWD = 2.0 ** -15
# sums over tokens and heads: fp32 in lanes, warps and CTAs, at most 2^-24 of the running
# magnitude for each of at most 4,096 additions that follow one another
DW = 2.0 ** -12


def inputs(L, H, seed, far=False):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(L, 3 * H * 128, generator=g) * torch.exp(0.5 * torch.randn(L, 1, generator=g))
    pos = torch.randint(-9, 60, (L, 3), generator=g, dtype=torch.int32)
    if far:
        pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (L, 3), generator=g).to(torch.int32)
    w = [1 + 0.3 * torch.randn(128, generator=g) for _ in range(2)]
    dout = torch.randn(L, 3 * H * 128, generator=g)
    return (qkv.to(torch.bfloat16).to(DEV), pos.to(DEV), w[0].to(DEV), w[1].to(DEV),
            dout.to(torch.bfloat16).to(DEV))


def banded(L, H):
    band = torch.full((L + 2, 3 * H * 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    return band, band[1:L + 1]


def bound(ref, big, share):
    return tr.U * ref.abs() + (1 + tr.U) * share * big + 2.0 ** -133


def norm(h3, qkv, pos, wq, wk, H, eps, **kw):
    L = qkv.shape[0]
    band, out = banded(L, H)
    h3.h3_qk_norm_mrope(qkv, pos, wq, wk, L, H, 128, eps, out, **kw)
    assert h3.h3_sync_status() == 0
    assert torch.isnan(band[0]).all() and torch.isnan(band[-1]).all()
    return out


def norm_bwd(h3, qkv, pos, wq, wk, dout, H, eps, **kw):
    L = qkv.shape[0]
    n = h3.h3_qk_norm_mrope_bwd_workspace_size(L, H)
    room = torch.full((n + 8192,), 0x5A, dtype=torch.uint8, device=DEV)
    band, out = banded(L, H)
    dw = torch.full((2, 132), float("nan"), device=DEV)
    h3.h3_qk_norm_mrope_bwd(qkv, pos, wq, wk, dout, L, H, 128, eps, room[4096:], n, out, dw[0, 1:129],
                            dw[1, 1:129], **kw)
    assert h3.h3_sync_status() == 0
    assert torch.isnan(band[0]).all() and torch.isnan(band[-1]).all()
    assert (room[:4096] == 0x5A).all() and (room[4096 + n:] == 0x5A).all()
    assert torch.isnan(dw[:, 0]).all() and torch.isnan(dw[:, 129:]).all()
    return out, dw[0, 1:129], dw[1, 1:129]


def check(h3, L, H, seed=0, eps=1e-6, weights=True, far=False, **kw):
    qkv, pos, wq, wk, dout = inputs(L, H, seed, far)
    if not weights:
        wq = wk = None
    ref, big = tr.qk_norm(qkv, pos, wq, wk, H, eps, **kw)
    got = norm(h3, qkv, pos, wq, wk, H, eps, **kw)
    tr.assert_within(got, ref, bound(ref, big, FWD), f"norm L={L} H={H}")
    d = H * 256
    assert torch.equal(got[:, d:], qkv[:, d:])
    refs, bigs = tr.qk_norm_bwd(qkv, pos, wq, wk, dout, H, eps, **kw)
    gots = norm_bwd(h3, qkv, pos, wq, wk, dout, H, eps, **kw)
    tr.assert_within(gots[0], refs[0], bound(refs[0], bigs[0], BWD), f"gradient L={L} H={H}")
    assert torch.equal(gots[0][:, d:], dout[:, d:])
    for i in (1, 2):
        tr.assert_within(gots[i], refs[i], DW * bigs[i] + 1e-30, f"dw {i} L={L} H={H}")


@pytest.mark.parametrize("L,H", [(1, 1), (1, 40), (1, 128), (2, 3), (7, 1), (31, 5), (64, 2), (129, 7),
                                 (300, 40), (1031, 16), (4099, 2), (20000, 1), (3001, 9)])
def test_shapes(h3, L, H):
    check(h3, L, H, seed=L + H)


@pytest.mark.parametrize("kw", [dict(sec=(128, 0, 0)), dict(sec=(0, 0, 128)), dict(sec=(2, 124, 2)),
                                dict(sec=(42, 44, 42)), dict(base=1e6), dict(base=1.5),
                                dict(base=0.01), dict(eps=0.0), dict(eps=0.5), dict(weights=False)])
def test_options(h3, kw):
    check(h3, 77, 3, seed=5, **kw)


def test_far_positions(h3):
    """Angles of positions up to 2^31: a frequency is kept to 2^-55 of a turn, so the angle is
    right to 2^-22 as for near ones (the definition in 64 bits loses 2^-53 of 2^31 radians)."""
    check(h3, 500, 2, seed=6, far=True)


def test_agrees_with_the_rotation_alone(h3):
    """Heads of unit mean square and no weights: what h3_mrope_apply gives, but for one rounding."""
    L, H = 200, 4
    qkv, pos, _, _, _ = inputs(L, H, 8)
    x = qkv.float().view(L, 3 * H, 128)
    qkv = (torch.sign(x) + (x == 0)).view(L, -1).to(torch.bfloat16)   # values of +-1
    turned = qkv.clone()
    h3.h3_mrope_apply(turned, pos, L, H)
    got = norm(h3, qkv, pos, None, None, H, 0.0)
    assert float((got.float() - turned.float()).abs().max()) <= 2 * 2.0 ** -8 * 2 ** 0.5


def test_in_place(h3):
    for L, H in ((1, 40), (333, 3)):
        qkv, pos, wq, wk, dout = inputs(L, H, 9)
        ref = norm(h3, qkv, pos, wq, wk, H, 1e-6)
        same = qkv.clone()
        h3.h3_qk_norm_mrope(same, pos, wq, wk, L, H, 128, 1e-6, same)
        gref, a, b = norm_bwd(h3, qkv, pos, wq, wk, dout, H, 1e-6)
        n = h3.h3_qk_norm_mrope_bwd_workspace_size(L, H)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        dsame, dwq, dwk = dout.clone(), torch.empty(128, device=DEV), torch.empty(128, device=DEV)
        h3.h3_qk_norm_mrope_bwd(qkv, pos, wq, wk, dsame, L, H, 128, 1e-6, ws, n, dsame, dwq, dwk)
        assert h3.h3_sync_status() == 0
        assert torch.equal(same, ref) and torch.equal(dsame, gref)
        # the warps' shares differ, so the sums' order may
        assert torch.allclose(dwq, a, rtol=1e-3, atol=1e-3) and torch.allclose(dwk, b, rtol=1e-3, atol=1e-3)


def test_weight_gradients_are_optional(h3):
    L, H = 100, 2
    qkv, pos, wq, wk, dout = inputs(L, H, 10)
    ref, a, b = norm_bwd(h3, qkv, pos, wq, wk, dout, H, 1e-6)
    n = h3.h3_qk_norm_mrope_bwd_workspace_size(L, H)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    for q, k in ((True, False), (False, True), (False, False)):
        out = torch.full_like(ref, float("nan"))
        dq = torch.full((128,), -7.0, device=DEV) if q else None
        dk = torch.full((128,), -7.0, device=DEV) if k else None
        h3.h3_qk_norm_mrope_bwd(qkv, pos, wq, wk, dout, L, H, 128, 1e-6, ws if q or k else None,
                                n if q or k else 0, out, dq, dk)
        assert h3.h3_sync_status() == 0
        assert torch.equal(out, ref)
        assert dq is None or torch.equal(dq, a)
        assert dk is None or torch.equal(dk, b)


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_heads_out_of_range_and_of_zeros(h3, eps):
    """Squares beyond fp32, or (eps aside) below it; heads of zeros; an infinity or a NaN stays
    in its head."""
    H, L = 2, 12
    qkv, pos, wq, wk, dout = inputs(L, H, 11)
    x = qkv.float().view(L, 3, H, 128)
    scales = [1e18, 1e30, 2.0 ** 120, 1e-18, 1e-25, 2.0 ** -120, 0.0, 1.0, 1e10, 1e-10, 1e-38, 1.0]
    for i, s in enumerate(scales):
        x[i, :2, 0] = (x[i, :2, 0] / x[i, :2, 0].abs().amax() * s)
    qkv = x.view(L, -1).to(torch.bfloat16)
    ref, big = tr.qk_norm(qkv, pos, wq, wk, H, eps)
    got = norm(h3, qkv, pos, wq, wk, H, eps)
    tr.assert_within(got, ref, bound(ref, big, FWD), "norm")
    refs, bigs = tr.qk_norm_bwd(qkv, pos, wq, wk, dout, H, eps)
    gots = norm_bwd(h3, qkv, pos, wq, wk, dout, H, eps)
    top = 3.3895e38                                    # gradients that bf16 cannot hold
    fine = (refs[0].abs() + bigs[0] * BWD).view(L, -1) < top
    assert fine.float().mean() > 0.9
    pick = lambda t: torch.where(fine, t.double(), torch.zeros_like(t.double()))  # noqa: E731
    tr.assert_within(pick(gots[0]), pick(refs[0]), bound(refs[0], bigs[0], BWD), "gradient")
    for i in (1, 2):
        tr.assert_within(gots[i], refs[i], DW * bigs[i] + 1e-30, f"dw {i}")
    # one bad value: its head alone
    bad = qkv.clone()
    bad[3, 5], bad[4, H * 128 + 128 + 9] = float("inf"), float("nan")
    other = norm(h3, bad, pos, wq, wk, H, eps)
    same = torch.ones_like(bad, dtype=torch.bool)
    same[3, :128] = False
    same[4, H * 128 + 128:H * 128 + 256] = False
    assert torch.equal(other[same], got[same])
    assert torch.isnan(other[3, 4:6]).any() and torch.isnan(other[4, H * 128 + 128:H * 128 + 256]).all()


def test_gradient_against_differences(h3):
    """sum(dout * y) along random directions: the formula's gradient (kernel) against central
    differences of the definition in 64 bits."""
    L, H, eps = 40, 2, 1e-6
    qkv, pos, wq, wk, dout = inputs(L, H, 12)
    d, dwq, dwk = norm_bwd(h3, qkv, pos, wq, wk, dout, H, eps)
    g = torch.Generator(device=DEV).manual_seed(3)
    f = lambda x, a, b: (tr.qk_norm(x, pos, a, b, H, eps)[0] * dout.double()).sum()  # noqa: E731
    _, bigs = tr.qk_norm_bwd(qkv, pos, wq, wk, dout, H, eps)
    for _ in range(4):
        u = torch.randn(qkv.shape, generator=g, device=DEV, dtype=torch.float64)
        uq, uk = torch.randn(2, 128, generator=g, device=DEV, dtype=torch.float64)
        t = 1e-6
        q, a, b = qkv.double(), wq.double(), wk.double()
        diff = (f(q + t * u, a + t * uq, b + t * uk) - f(q - t * u, a - t * uq, b - t * uk)) / (2 * t)
        got = (d.double() * u).sum() + (dwq.double() * uq).sum() + (dwk.double() * uk).sum()
        off = ((tr.U * d.double().abs() + BWD * bigs[0]) * u.abs()).sum()
        off += DW * ((bigs[1] * uq.abs()).sum() + (bigs[2] * uk.abs()).sum())
        assert abs(float(diff - got)) <= float(off) + 1e-5 * abs(float(diff))


def test_same_bits_streams_and_graphs(h3):
    L, H = 2000, 4
    qkv, pos, wq, wk, dout = inputs(L, H, 13)
    ref = norm(h3, qkv, pos, wq, wk, H, 1e-6)
    gref, a, b = norm_bwd(h3, qkv, pos, wq, wk, dout, H, 1e-6)
    n = h3.h3_qk_norm_mrope_bwd_workspace_size(L, H)

    def call(o, ws, out, dq, dk, stream=None):
        h3.h3_qk_norm_mrope(qkv, pos, wq, wk, L, H, 128, 1e-6, o, stream=stream)
        h3.h3_qk_norm_mrope_bwd(qkv, pos, wq, wk, dout, L, H, 128, 1e-6, ws, n, out, dq, dk, stream=stream)

    sets = [(torch.empty_like(ref), torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty_like(ref),
             torch.empty(128, device=DEV), torch.empty(128, device=DEV)) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, t in zip(streams, sets):
        call(*t, stream=s)
    streams[0].synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(streams[0]), torch.cuda.graph(g, stream=streams[0]):
        call(*sets[2])
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert h3.h3_sync_status() == 0
    for o, _, out, dq, dk in sets:
        assert torch.equal(o, ref) and torch.equal(out, gref)
        assert torch.equal(dq, a) and torch.equal(dk, b)


def test_offsets_past_32_bits(h3):
    L, H = 290_000, 40
    qkv = torch.zeros(L, 3 * H * 128, dtype=torch.bfloat16, device=DEV)
    assert qkv.numel() > 2 ** 32
    g = torch.Generator(device=DEV).manual_seed(1)
    tail = 100
    qkv[-tail:].copy_(torch.randn(tail, 3 * H * 128, generator=g, device=DEV))
    pos = torch.arange(3 * L, device=DEV, dtype=torch.int32).view(L, 3).contiguous()
    wq, wk = (1 + 0.1 * torch.randn(128, generator=g, device=DEV) for _ in range(2))
    out = torch.empty_like(qkv)
    h3.h3_qk_norm_mrope(qkv, pos, wq, wk, L, H, 128, 1e-6, out)
    assert h3.h3_sync_status() == 0
    ref, big = tr.qk_norm(qkv[-tail:], pos[-tail:], wq, wk, H, 1e-6)
    tr.assert_within(out[-tail:], ref, bound(ref, big, FWD), "last tokens")
    n = h3.h3_qk_norm_mrope_bwd_workspace_size(L, H)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    dwq, dwk = torch.empty(128, device=DEV), torch.empty(128, device=DEV)
    h3.h3_qk_norm_mrope_bwd(qkv, pos, wq, wk, out, L, H, 128, 1e-6, ws, n, out, dwq, dwk)
    assert h3.h3_sync_status() == 0
    refs, bigs = tr.qk_norm_bwd(qkv[-tail:], pos[-tail:], wq, wk, ref.to(torch.bfloat16), H, 1e-6)
    # dout is the stored output: one rounding of it more
    tr.assert_within(out[-tail:], refs[0], bound(refs[0], bigs[0], BWD + 2 * tr.U), "last tokens' gradient")
    for got, r, m in ((dwq, refs[1], bigs[1]), (dwk, refs[2], bigs[2])):
        tr.assert_within(got, r, (DW + 2 * tr.U) * m, "dw")


@pytest.mark.parametrize("L,H", [(1, 1), (1, 40), (130, 3), (5000, 2)])
def test_checked_build_reports_nothing(h3, checked, L, H):  # noqa: F811
    qkv, pos, wq, wk, dout = inputs(L, H, L)

    def run():
        n = h3lib.h3_qk_norm_mrope_bwd_workspace_size(L, H)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        a, b = torch.empty_like(qkv), torch.empty_like(qkv)
        dq, dk = torch.empty(128, device=DEV), torch.empty(128, device=DEV)
        h3lib.h3_qk_norm_mrope(qkv, pos, wq, wk, L, H, 128, 1e-6, a)
        h3lib.h3_qk_norm_mrope_bwd(qkv, pos, wq, wk, dout, L, H, 128, 1e-6, ws, n, b, dq, dk)
        return a, b, dq, dk

    _both(checked, run)
