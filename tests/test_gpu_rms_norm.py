"""RMS norm with the residual's addition and an E4M3 or 4-bit output, against the definition
in 64 bits.

The norm is of the stored sum, whose bits equal bf16(fp32(x + res)).  y = sum * weight * rstd
in fp32: the sum of squares is joined from chains of at most 8 terms by at most 14 pairwise
additions (22 roundings, halved by the square root), the inverse square root is within two
steps (2^-22), the mean and eps take 2 more and the two products 2: y is within
(13 + 4 + 2) 2^-24 < 2^-19 of its value.  What is rounded to a grid may therefore differ from
the definition's by half a step of the grid plus 2^-18 of the value (the quantiser's own
products included)."""
import math

import numpy as np
import pytest
import torch

from tests import _fp4 as f4
from tests._fp8 import e4m3_decode
from tests._parity import to64
from tests.test_gpu_fp4 import CANARY, _assert_product, _guarded, _intact, _quant

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
SLACK = 2.0 ** -18


def _inputs(L, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(L, d, generator=g) * torch.exp2(torch.randint(-8, 9, (L, 1), generator=g).float())
    res = torch.randn(L, d, generator=g) * torch.exp2(torch.randint(-8, 9, (L, 1), generator=g).float())
    w = 1.0 + 0.3 * torch.randn(d, generator=g)
    if L > 4:
        x[1] = 0.0
        res[1] = 0.0                      # a row of zeros: y = 0
        res[2] = -x[2].to(torch.bfloat16).float()   # and one that cancels
        x[3, : d // 2] *= 2.0 ** -12
    w[5] = 0.0
    return x.to(torch.bfloat16), res.to(torch.bfloat16), w


def _reference(x, res, w):
    s = x if res is None else (x.float() + res.float()).to(torch.bfloat16)
    f = to64(s)
    return s, f / np.sqrt((f * f).mean(axis=1, keepdims=True) + EPS) * to64(w)


def _check_fp8(q, scale, y):
    amax = np.abs(y).max(axis=1)
    want = np.where(amax > 0, amax / 448.0, 1.0)
    assert np.all(np.abs(scale - want) <= SLACK * want)
    t = y / scale[:, None]
    # half a step of E4M3: 2^-4 of the power of two below |t|, at least 2^-10
    step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(t), 2.0 ** -20))) - 4.0), 2.0 ** -10)
    assert np.all(np.abs(e4m3_decode(q) - t) <= step + SLACK * np.abs(t))


SHAPES = [(1, 128), (1, 5120), (5, 256), (33, 640), (128, 2048), (301, 1152), (257, 5120), (19, 8192),
          (13, 16384), (3000, 384)]


@pytest.mark.parametrize("L,d", SHAPES)
@pytest.mark.parametrize("with_res", [True, False])
def test_norm_fp8(h3, L, d, with_res):
    x, res, w = _inputs(L, d, L + d)
    res = res if with_res else None
    gs, s = _guarded(L * d * 2)
    gq, q = _guarded(L * d)
    gc, sc = _guarded(L * 4)
    dv = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    h3.h3_rms_norm_fp8(dv(x), dv(res), dv(w), L, d, EPS, s, q, sc)
    assert h3.h3_sync_status() == 0
    _intact(gs, gq, gc)
    want, y = _reference(x, res, w)
    assert torch.equal(s.view(torch.bfloat16).view(L, d).cpu().view(torch.int16), want.view(torch.int16))
    _check_fp8(q.view(L, d).cpu().numpy(), sc.view(torch.float32).cpu().numpy().astype(np.float64), y)
    # without the sum's output, and with the sum in place of the residual (or of x)
    q2, sc2 = torch.empty_like(q), torch.empty_like(sc)
    h3.h3_rms_norm_fp8(dv(x), dv(res), dv(w), L, d, EPS, None, q2, sc2.view(torch.float32))
    assert torch.equal(q2, q) and torch.equal(sc2, sc)
    xin, rin = dv(x), dv(res)
    h3.h3_rms_norm_fp8(xin, rin, dv(w), L, d, EPS, rin if with_res else xin, q2, sc2.view(torch.float32))
    assert h3.h3_sync_status() == 0
    assert torch.equal(q2, q) and torch.equal(sc2, sc)
    assert torch.equal((rin if with_res else xin).cpu().view(torch.int16), want.view(torch.int16))


def test_sum_in_place_of_x_and_the_same_tensor_twice(h3):
    L, d = 37, 640
    x, res, w = _inputs(L, d, 9)
    for same in (False, True):
        xin = x.to(DEV)
        rin = xin if same else res.to(DEV)
        want, y = _reference(x, x if same else res, w)
        q = torch.empty(L, d, dtype=torch.uint8, device=DEV)
        sc = torch.empty(L, device=DEV)
        h3.h3_rms_norm_fp8(xin, rin, w.to(DEV), L, d, EPS, xin, q, sc)
        assert h3.h3_sync_status() == 0
        assert torch.equal(xin.cpu().view(torch.int16), want.view(torch.int16))
        _check_fp8(q.cpu().numpy(), to64(sc), y)
        if not same:
            assert torch.equal(rin.cpu().view(torch.int16), res.view(torch.int16))


@pytest.mark.parametrize("fmt", [f4.MX, f4.NV])
@pytest.mark.parametrize("L,d", SHAPES)
def test_norm_fp4(h3, fmt, L, d):
    x, res, w = _inputs(L, d, L + d + fmt)
    S = d // f4.BLOCK[fmt]
    n = h3.h3_fp4_scale_bytes(fmt, L, d)
    gs, s = _guarded(L * d * 2)
    gq, q = _guarded(L * d // 2)
    gb, bs = _guarded(n)
    row = torch.ones(L, device=DEV)
    h3.h3_rms_norm_fp4(x.to(DEV), res.to(DEV), w.to(DEV), L, d, EPS, fmt, s, q, bs,
                       row if fmt == f4.NV else None)
    assert h3.h3_sync_status() == 0
    _intact(gs, gq, gb)
    want, y = _reference(x, res, w)
    assert torch.equal(s.view(torch.bfloat16).view(L, d).cpu().view(torch.int16), want.view(torch.int16))
    flat = bs.cpu().numpy()
    keep = np.ones(flat.size, dtype=bool)
    keep[f4.scale_index(L, S)] = False
    assert np.all(flat[keep] == CANARY)
    byte = f4.untile(flat, L, S)
    r = row.cpu().numpy().astype(np.float64)
    a = np.abs(y).reshape(L, S, -1).max(axis=2)
    sv = f4.scale_values(byte, fmt)
    if fmt == f4.MX:
        # the smallest power of two with a <= 6 scale, on a within SLACK of the definition's
        assert np.all(a <= 6.0 * sv * (1 + SLACK))
        assert np.all((a > 3.0 * sv * (1 - SLACK)) | (byte == 0))
    else:
        top = a.max(axis=1)
        assert np.all(top <= 2688.0 * r * (1 + SLACK))
        assert np.all((top > 1344.0 * r * (1 - SLACK)) | (top == 0))
        t = a / (6.0 * r[:, None])
        step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(t, 2.0 ** -20))) - 4.0), 2.0 ** -10)
        assert np.all(np.abs(sv - np.minimum(t, 448.0)) <= step + SLACK * t)
    full = (sv * r[:, None]).repeat(f4.BLOCK[fmt], axis=1)
    live = full > 0
    t = np.where(live, y / np.where(live, full, 1.0), 0.0)
    got = f4.e2m1_decode(f4.unpack(q.view(L, d // 2).cpu().numpy()))
    assert np.all(got[~live] == 0.0)
    clipped = np.clip(t, -6.0, 6.0)
    assert np.all(np.abs(got - clipped) <= f4.half_step(clipped) + SLACK * np.abs(t))
    # the same bits again, the sum in place of the residual
    rin, q2, bs2, row2 = res.to(DEV), torch.empty_like(q), torch.empty_like(bs), torch.ones(L, device=DEV)
    bs2.fill_(CANARY)
    h3.h3_rms_norm_fp4(x.to(DEV), rin, w.to(DEV), L, d, EPS, fmt, rin, q2, bs2,
                       row2 if fmt == f4.NV else None)
    assert h3.h3_sync_status() == 0
    assert torch.equal(q2, q) and torch.equal(bs2, bs) and torch.equal(row2, row)


def test_rows_of_tiny_values_and_weights(h3):
    """Rows whose largest value is so small that 448 / max would leave fp32: finite codes, and
    the scale's lower bound."""
    L, d = 4, 256
    x = torch.zeros(L, d)
    x[0], x[1, ::3], x[2] = 2.0 ** -120, 2.0 ** -133, 1.0
    w = torch.ones(d)
    w[:128] = 2.0 ** -125
    for eps in (EPS, 1.0):
        q = torch.empty(L, d, dtype=torch.uint8, device=DEV)
        sc = torch.empty(L, device=DEV)
        h3.h3_rms_norm_fp8(x.to(torch.bfloat16).to(DEV), None, w.to(DEV), L, d, eps, None, q, sc)
        assert h3.h3_sync_status() == 0
        f = to64(x.to(torch.bfloat16))
        y = f / np.sqrt((f * f).mean(axis=1, keepdims=True) + eps) * to64(w)
        s = sc.cpu().numpy().astype(np.float64)
        amax = np.abs(y).max(axis=1)
        want = np.where(amax > 0, np.maximum(amax / 448.0, 2.0 ** -126), 1.0)
        assert np.all(np.abs(s - want) <= SLACK * want)
        t = y / s[:, None]
        got = e4m3_decode(q.cpu().numpy())
        step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(t), 2.0 ** -20))) - 4.0), 2.0 ** -10)
        # y itself may be below the normal numbers: rounded to a multiple of 2^-149
        assert np.all(np.abs(got - t) <= step + SLACK * np.abs(t) + 2.0 ** -149 / s[:, None])


def test_offsets_past_32_bits(h3):
    """2.3e9 elements: sampled rows, the last ones among them."""
    L, d = 450_001, 5120
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.empty(L, d, dtype=torch.bfloat16, device=DEV)
    for r in range(0, L, 50_000):
        n = min(50_000, L - r)
        x[r:r + n] = torch.randn(n, d, generator=g, device=DEV)
    res = x.flip(0)
    w = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
    rows = torch.tensor([0, 1, 2 ** 31 // d, 2 ** 31 // d + 1, L - 2, L - 1, 77_777, 300_000], device=DEV)
    want, y = _reference(x[rows].cpu(), res[rows].cpu(), w.cpu())
    q = torch.empty(L, d, dtype=torch.uint8, device=DEV)
    sc = torch.empty(L, device=DEV)
    h3.h3_rms_norm_fp8(x, res, w, L, d, EPS, res, q, sc)
    assert h3.h3_sync_status() == 0
    assert torch.equal(res[rows].cpu().view(torch.int16), want.view(torch.int16))
    _check_fp8(q[rows].cpu().numpy(), to64(sc[rows]), y)


@pytest.mark.parametrize("L", [1, 40])
def test_nonfinite_values_stay_visible(h3, L):
    d = 512
    x = torch.randn(L, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[L // 2, 100] = float("nan")
    w = torch.ones(d, device=DEV)
    q = torch.empty(L, d, dtype=torch.uint8, device=DEV)
    sc = torch.empty(L, device=DEV)
    h3.h3_rms_norm_fp8(x.to(DEV), None, w, L, d, EPS, None, q, sc)
    bad = ((q & 0x7F) == 0x7F).cpu()
    assert bool(bad[L // 2].all()) and int(bad.any(dim=1).sum()) == 1
    for fmt in (f4.MX, f4.NV):
        bs = torch.empty(h3.h3_fp4_scale_bytes(fmt, L, d), dtype=torch.uint8, device=DEV)
        y = torch.empty(L, d, dtype=torch.bfloat16, device=DEV)
        h3.h3_rms_norm_fp4(x.to(DEV), None, w, L, d, EPS, fmt, None, q, bs, sc)
        h3.h3_dequantize_rows_fp4(q, bs, sc if fmt == f4.NV else None, fmt, L, d, y)
        assert h3.h3_sync_status() == 0
        bad = torch.isnan(y).cpu()
        assert bool(bad[L // 2].all()) and int(bad.any(dim=1).sum()) == 1


@pytest.mark.parametrize("L", [1, 21, 400])
def test_norm_product_norm_product(h3, L):
    """Two layers' worth of a pre-norm stream as it would be used: norm into 4 bits, product,
    norm of the sum into 8 bits, product; each stage against the definition from the stage
    before it as the GPU stored it."""
    d, fmt = 768, f4.NV
    g = torch.Generator().manual_seed(L)
    x = torch.randn(L, d, generator=g).to(torch.bfloat16).to(DEV)
    stream = torch.randn(L, d, generator=g).to(torch.bfloat16).to(DEV)
    w1, w2 = ((1.0 + 0.1 * torch.randn(d, generator=g)).to(DEV) for _ in range(2))
    W = (torch.randn(d, d, generator=g) / math.sqrt(d)).to(torch.bfloat16)
    qW = _quant(h3, W.to(DEV), fmt)
    q = torch.empty(L, d // 2, dtype=torch.uint8, device=DEV)
    bs = torch.zeros(h3.h3_fp4_scale_bytes(fmt, L, d), dtype=torch.uint8, device=DEV)
    s = torch.empty(L, device=DEV)
    h3.h3_rms_norm_fp4(x, stream, w1, L, d, EPS, fmt, stream, q, bs, s)
    out = torch.empty(L, d, dtype=torch.bfloat16, device=DEV)
    h3.h3_gemm_fp4(q, bs, s, *qW, fmt, L, d, d, out)
    first = stream.clone()
    q8 = torch.empty(L, d, dtype=torch.uint8, device=DEV)
    s8 = torch.empty(L, device=DEV)
    h3.h3_rms_norm_fp8(out, stream, w2, L, d, EPS, stream, q8, s8)
    W8, W8s = torch.empty(d, d, dtype=torch.uint8, device=DEV), torch.empty(d, device=DEV)
    h3.h3_quantize_rows_fp8(W.to(DEV), d, d, W8, W8s)
    out2 = torch.empty_like(out)
    h3.h3_gemm_fp8(q8, s8, W8, W8s, L, d, d, out2)
    assert h3.h3_sync_status() == 0
    S = d // f4.BLOCK[fmt]
    a = f4.values(f4.unpack(q.cpu().numpy()), f4.untile(bs.cpu().numpy(), L, S), s.cpu().numpy(), fmt)
    _assert_product(out, a, f4.dequant(to64(W), fmt), d, "first product")
    want, y = _reference(out.cpu(), first.cpu(), w2.cpu())
    assert torch.equal(stream.cpu().view(torch.int16), want.view(torch.int16))
    _check_fp8(q8.cpu().numpy(), to64(s8), y)
    a8 = e4m3_decode(q8.cpu().numpy()) * to64(s8)[:, None]
    b8 = e4m3_decode(W8.cpu().numpy()) * to64(W8s)[:, None]
    _assert_product(out2, a8, b8, d, "second product")
