"""RMS norm of rows whose squares leave fp32, and of rows of zeros without an eps.

The norm of a row is that of the row times a power of two, with eps times its square; taken
with a power from the row's largest value every square that matters is an ordinary number.
The sum of such a row joins 8 squares, at most 4 of those, 32 lanes and at most 16 warps, one
after the other (60 roundings, halved by the square root); the inverse square root is within
two steps (4 x 2^-24), the mean and eps take 2 more, the two products 2 and the quantiser 4:
42 x 2^-24, below 2^-18.  (The sum of an ordinary row: chains of 8 squares, 2 pairs, 5 steps
over the lanes, at most 15 over the warps, 30 roundings.)  SLACK = 2^-18 covers both, and the
inverse square root of the largest rows, which is short of two bits."""
import numpy as np
import pytest
import torch

from tests import _fp4 as f4
from tests._parity import to64
from tests.test_gpu_rms_norm import SLACK, _check_fp8

pytestmark = pytest.mark.gpu
DEV = "cuda"
# bf16 rows of every size: ordinary ones between those whose squares overflow or vanish
EXPS = [0, 126, 100, 64, 63, 40, -1, -40, -62, -63, -64, -75, -100, -126, -132]
# d: one, two, four or more warps a row, one to four rows a CTA, the widest
WIDTHS = [128, 512, 640, 1152, 2048, 5120, 16384]


def _rows(d, seed):
    g = torch.Generator().manual_seed(seed)
    L = 2 * len(EXPS) + 5
    x = torch.randn(L, d, generator=g)
    x = x.clamp(-3.0, 3.0) / 4.0 + 0.1
    for i in range(L):
        x[i] *= 2.0 ** EXPS[i % len(EXPS)]
    x[3] = 0.0
    x[4, :] = 0.0
    x[4, d - 1] = 2.0 ** -133            # the smallest bf16 alone
    x[9, : d // 2] *= 2.0 ** -80         # halves of different size
    x[-1] = x[-1].sign() * 3.3895313892515355e38
    w = 1.0 + 0.3 * torch.randn(d, generator=g)
    return x.to(torch.bfloat16), w


def _definition(x, w, eps):
    """y in 64 bits; a row of zeros is zeros."""
    f, e = to64(x), float(np.float32(eps))
    ms = (f * f).mean(axis=1, keepdims=True) + e
    return np.where(f == 0, 0.0, f / np.sqrt(np.where(ms > 0, ms, 1.0)) * to64(w))


@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-38, 1e-30, 1e-6])
@pytest.mark.parametrize("d", WIDTHS)
def test_rows_of_any_size_to_e4m3(h3, d, eps):
    x, w = _rows(d, d)
    L = x.shape[0]
    y = _definition(x, w, eps)
    for with_res in (False, True):
        # x + res of two halves is x again
        half = (to64(x) / 2).astype(np.float32)
        res = torch.from_numpy(half).to(torch.bfloat16) if with_res else None
        a = (x.float() - res.float()).to(torch.bfloat16) if with_res else x
        if with_res:
            s64 = (a.float() + res.float()).to(torch.bfloat16)
            y = _definition(s64, w, eps)
        q = torch.empty(L, d, dtype=torch.uint8, device=DEV)
        sc = torch.empty(L, device=DEV)
        s = torch.empty(L, d, dtype=torch.bfloat16, device=DEV)
        h3.h3_rms_norm_fp8(a.to(DEV), None if res is None else res.to(DEV), w.to(DEV), L, d, eps, s, q, sc)
        assert h3.h3_sync_status() == 0
        want = s64 if with_res else x
        assert torch.equal(s.cpu().view(torch.int16), want.view(torch.int16))     # stored as it is
        scale = to64(sc)
        codes = q.cpu().numpy()
        assert not np.any((codes & 0x7F) == 0x7F)
        # rows so small beside eps that the scale meets its lower bound: eps 1e-6 and 2^-133 alone
        small = np.abs(y).max(axis=1) / 448.0 < 2.0 ** -126 * (1 + SLACK)
        assert np.all(scale[small & (np.abs(y).max(axis=1) > 0)] == np.float32(2.0 ** -126))
        _check_fp8(codes[~small], scale[~small], y[~small])
        # the same bits with the sum in place of an input, and without it
        for target in ("x", "res", None):
            if target == "res" and res is None:
                continue
            ax, rx = a.to(DEV), None if res is None else res.to(DEV)
            q2, sc2 = torch.empty_like(q), torch.empty_like(sc)
            h3.h3_rms_norm_fp8(ax, rx, w.to(DEV), L, d, eps, {"x": ax, "res": rx, None: None}[target], q2, sc2)
            assert h3.h3_sync_status() == 0
            assert torch.equal(q2, q) and torch.equal(sc2, sc)
        zero = np.abs(y).max(axis=1) == 0
        assert zero.any() and np.all(scale[zero] == 1.0) and np.all(codes[zero] & 0x7F == 0)


@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-6])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("fmt", [f4.MX, f4.NV])
def test_rows_of_any_size_to_four_bits(h3, fmt, d, eps):
    """What the 4-bit rows stand for is within half a step of y (and of the E4M3 rounding of
    the scale, which may clip by 2^-4)."""
    x, w = _rows(d, d + fmt)
    L, S, blk = x.shape[0], d // f4.BLOCK[fmt], f4.BLOCK[fmt]
    y = _definition(x, w, eps)
    q = torch.empty(L, d // 2, dtype=torch.uint8, device=DEV)
    bs = torch.zeros(h3.h3_fp4_scale_bytes(fmt, L, d), dtype=torch.uint8, device=DEV)
    row = torch.ones(L, device=DEV)
    h3.h3_rms_norm_fp4(x.to(DEV), None, w.to(DEV), L, d, eps, fmt, None, q, bs,
                       row if fmt == f4.NV else None)
    assert h3.h3_sync_status() == 0
    byte, r = f4.untile(bs.cpu().numpy(), L, S), to64(row)
    sv = f4.scale_values(byte, fmt) * r[:, None]
    assert np.all(np.isfinite(sv))
    a = np.abs(y).reshape(L, S, blk).max(axis=2)
    if fmt == f4.MX:
        assert np.all(a <= 6.0 * sv * (1 + SLACK))
        assert np.all((a > 3.0 * sv * (1 - SLACK)) | (byte == 0))
    else:
        top = a.max(axis=1)
        low = r == 2.0 ** -117
        assert np.all(top <= 2688.0 * r * (1 + SLACK))
        assert np.all((top > 1344.0 * r * (1 - SLACK)) | (top == 0) | low)
        assert np.all(r[top == 0] == 1.0)
    full = sv.repeat(blk, axis=1)
    live = full > 0
    t = np.where(live, y / np.where(live, full, 1.0), 0.0)
    got = f4.e2m1_decode(f4.unpack(q.cpu().numpy()))
    assert np.all(got[~live] == 0.0)
    clipped = np.clip(t, -6.0, 6.0)
    # y may itself be below the normal numbers: off by 2^-149
    tiny = np.where(live, 2.0 ** -149 / np.where(live, full, 1.0), 0.0)
    assert np.all(np.abs(got - clipped) <= f4.half_step(clipped) + SLACK * np.abs(t) + tiny)


@pytest.mark.parametrize("d", [256, 2048, 5120])
def test_infinities_and_nans_among_large_rows(h3, d):
    """A row with a NaN stays NaN, a row with an infinity keeps the formula's zeros and NaN, and
    the rows beside them are those of the call without."""
    x, w = _rows(d, 3)
    L = x.shape[0]
    bad = x.clone()
    bad[1, 7], bad[6, 9], bad[12, d - 1] = float("nan"), float("inf"), -float("inf")
    out = []
    for v in (x, bad):
        q = torch.empty(L, d, dtype=torch.uint8, device=DEV)
        sc = torch.empty(L, device=DEV)
        h3.h3_rms_norm_fp8(v.to(DEV), None, w.to(DEV), L, d, 0.0, None, q, sc)
        assert h3.h3_sync_status() == 0
        out.append((q.cpu(), sc.cpu()))
    keep = torch.ones(L, dtype=torch.bool)
    keep[[1, 6, 12]] = False
    assert torch.equal(out[0][0][keep], out[1][0][keep]) and torch.equal(out[0][1][keep], out[1][1][keep])
    nan = (out[1][0] & 0x7F) == 0x7F
    assert bool(nan[1].all())
    for r, c in ((6, 9), (12, d - 1)):
        assert bool(nan[r, c]) and int(nan[r].sum()) == 1
        assert bool(((out[1][0][r] & 0x7F) == 0)[torch.arange(d) != c].all())
