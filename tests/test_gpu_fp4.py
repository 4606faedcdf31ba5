"""Microscaled 4-bit rows and their product on the GPU against the definitions in 64 bits.

Quantisation: codes, scales and row factors equal the definition's bit for bit (every step
but the two roundings is exact).  Product: E2M1 products under power-of-two or 4-bit scales
are exact in fp32, so an output differs from the exact sum of the operands' values by the
bf16 rounding of the result, half a step = 2^-8 of it, and by the fp32 additions: at most
one for each product and 64-column step, K + K / 64 + 1 roundings or truncations of a partial
sum, each at most 2^-23 of sum |a b|."""
import math

import numpy as np
import pytest
import torch

import oracle as orc
from h3inputs import CONFIGS
from tests import _fp4 as f4
from tests._parity import BF16_U, assert_parity, to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMTS = [f4.MX, f4.NV]
CANARY = 0xA5


def _guarded(nbytes):
    """A buffer of nbytes between two canary bands of 4 KB, and its middle."""
    b = torch.full((nbytes + 8192,), CANARY, dtype=torch.uint8, device=DEV)
    return b, b[4096:4096 + nbytes]


def _intact(*bufs):
    for b in bufs:
        assert bool((b[:4096] == CANARY).all()) and bool((b[-4096:] == CANARY).all())


def _quant(h3, x, fmt):
    """(codes, scale bytes, row factors, buffers) of x bf16 on the GPU."""
    R, K = x.shape
    n = h3.h3_fp4_scale_bytes(fmt, R, K)
    gq, q = _guarded(R * K // 2)
    gb, bs = _guarded(n)
    gs, s = _guarded(R * 4)
    h3.h3_quantize_rows_fp4(x, fmt, R, K, q, bs, s if fmt == f4.NV else None)
    assert h3.h3_sync_status() == 0
    _intact(gq, gb, gs)
    s = s.view(torch.float32)
    return q.view(R, K // 2), bs, (s if fmt == f4.NV else None)


def _wide_range(R, K, seed):
    """bf16 rows of every size, with zeros, ties and subnormals among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, K, generator=g) * torch.exp2(torch.randint(-30, 30, (R, 1), generator=g).float())
    x *= torch.exp2(torch.randint(-6, 7, (1, K), generator=g).float())
    x[torch.rand(R, K, generator=g) < 0.1] = 0.0
    if R > 8:
        # small whole numbers: quotients that are ties occur in every block
        x[1] = torch.randint(-14, 15, (K,), generator=g).float()
        x[2] = torch.randint(-2688, 2689, (K,), generator=g).float()
        x[3] = 0.0
        x[4] = 0.0
        x[4, 5] = 2.0 ** -133                       # the smallest bf16
        x[5] = x[5].sign() * 3.3895313892515355e38  # the largest
        x[6, :] = -0.0
        x[7] *= 2.0 ** -100
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,K", [(1, 128), (3, 256), (37, 384), (129, 640), (300, 5120), (66, 8320),
                                 (17, 20480), (9, 65536)])
def test_quantiser_equals_the_definition(h3, fmt, R, K):
    x = _wide_range(R, K, R + K + fmt)
    q, bs, s = _quant(h3, x.to(DEV), fmt)
    code, byte, row = f4.quantize(to64(x), fmt)
    S = K // f4.BLOCK[fmt]
    assert np.array_equal(f4.untile(bs.cpu().numpy(), R, S), byte)
    if fmt == f4.NV:
        assert np.array_equal(s.cpu().numpy().astype(np.float64), row)
    got = f4.unpack(q.cpu().numpy())
    assert np.array_equal(f4.e2m1_decode(got), f4.e2m1_decode(code))
    # the scale bytes of rows past the last are left as they were
    keep = np.ones(bs.numel(), dtype=bool)
    keep[f4.scale_index(R, S)] = False
    assert np.all(bs.cpu().numpy()[keep] == CANARY)
    # and back: exact in bf16, but for values below its normal range and for those that the
    # rounding took past its largest (the code 4 under the scale 2^126 is 2^128): infinity
    y = torch.full((R, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    h3.h3_dequantize_rows_fp4(q, bs, s, fmt, R, K, y)
    assert h3.h3_sync_status() == 0
    want = f4.values(code, byte, row, fmt)
    got = to64(y)
    beyond = np.abs(want) >= 2.0 ** 127 * (2.0 - 2.0 ** -8)
    assert np.array_equal(got[beyond], np.copysign(np.inf, want[beyond]))
    got, want = got[~beyond], want[~beyond]
    assert np.all(np.abs(got - want) <= 2.0 ** -134)
    assert np.array_equal(got[np.abs(want) >= 2.0 ** -126], want[np.abs(want) >= 2.0 ** -126])


@pytest.mark.parametrize("fmt", FMTS)
def test_nonfinite_blocks_stand_for_nan(h3, fmt):
    R, K, blk = 6, 256, f4.BLOCK[fmt]
    x = torch.randn(R, K, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    clean = x.clone()
    x[1, 5], x[2, 40], x[3, K - 1] = float("nan"), float("inf"), -float("inf")
    q, bs, s = _quant(h3, x.to(DEV), fmt)
    y = torch.empty(R, K, dtype=torch.bfloat16, device=DEV)
    h3.h3_dequantize_rows_fp4(q, bs, s, fmt, R, K, y)
    got = to64_nan(y)
    bad = np.zeros((R, K), dtype=bool)
    for r, c in ((1, 5), (2, 40), (3, K - 1)):
        bad[r, c // blk * blk:(c // blk + 1) * blk] = True
    assert np.array_equal(np.isnan(got), bad)
    # the other blocks are those of the row without the bad ones
    clean[torch.from_numpy(bad)] = 0.0
    assert np.array_equal(got[~bad], f4.dequant(to64(clean), fmt)[~bad])


def to64_nan(t):
    return t.float().cpu().double().numpy()


def test_dequantiser_takes_any_scale_and_row_factor(h3):
    rng = np.random.default_rng(8)
    R, K = 140, 256
    for fmt in FMTS:
        S = K // f4.BLOCK[fmt]
        code = rng.integers(0, 16, (R, K)).astype(np.uint8)
        byte = rng.integers(0, 256 if fmt == f4.MX else 127, (R, S)).astype(np.uint8)
        if fmt == f4.NV:
            byte[3, 2] = 0x7F
        row = rng.uniform(0.5, 2.0, R).astype(np.float32)
        dv = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
        for s in (None, row):
            y = torch.empty(R, K, dtype=torch.bfloat16, device=DEV)
            h3.h3_dequantize_rows_fp4(dv(f4.pack(code)), dv(f4.tile(byte, 0x55)),
                                      None if s is None else dv(s), fmt, R, K, y)
            assert h3.h3_sync_status() == 0
            want = f4.values(code, byte, np.ones(R) if s is None else s, fmt)
            got = to64_nan(y)
            assert np.array_equal(np.isnan(got), np.isnan(want))
            ok = ~np.isnan(want) & (np.abs(want) < 3.3e38)
            # one rounding of the product with the row factor (2^-24), one to bf16
            assert np.all(np.abs(got - want)[ok] <= (BF16_U + 2.0 ** -23) * np.abs(want[ok]) + 2.0 ** -134)


def _product(h3, A, B, fmt, M, N, K):
    gc, c = _guarded(M * N * 2)
    c = c.view(torch.bfloat16)
    c.fill_(float("nan"))
    h3.h3_gemm_fp4(A[0], A[1], A[2], B[0], B[1], B[2], fmt, M, N, K, c)
    assert h3.h3_sync_status() == 0
    _intact(gc)
    return c.view(M, N)


def _assert_product(C, a, b, K, what):
    ref = a @ b.T
    mag = np.abs(a) @ np.abs(b).T
    err = np.abs(to64(C) - ref)
    assert np.all(np.isfinite(err)), what
    bound = BF16_U * np.abs(ref) + (K + K // 64 + 1) * 2.0 ** -23 * mag
    worst = float(np.max(err - bound))
    assert worst <= 0.0, f"{what}: {worst:.3e} over the bound"
    assert_parity(to64(C), ref, what)


SHAPES = [(1, 128, 128), (24, 39040, 128), (48, 512, 640), (49, 512, 640), (49, 384, 8320),
          (64, 256, 8192), (64, 256, 8064), (1, 12160, 256), (1, 12288, 256), (2, 5120, 2048),
          (2, 2560, 5120), (1, 6144, 4608), (1, 6144, 4736), (1, 256, 256), (2, 384, 384),
          (1, 5120, 2048), (3, 640, 1152), (4, 256, 4096), (5, 256, 1280), (7, 1280, 640),
          (16, 128, 2048), (33, 512, 384), (127, 128, 512), (128, 256, 1024), (129, 384, 1152),
          (257, 512, 512), (300, 640, 4096), (513, 256, 8192), (1000, 2048, 2048),
          (221, 5120, 640), (2049, 1024, 896)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_against_the_exact_sum(h3, fmt, M, N, K):
    g = torch.Generator().manual_seed(M + N + K)
    a = (torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).to(torch.bfloat16)
    b = (torch.randn(N, K, generator=g) / math.sqrt(K)).to(torch.bfloat16)
    C = _product(h3, _quant(h3, a.to(DEV), fmt), _quant(h3, b.to(DEV), fmt), fmt, M, N, K)
    _assert_product(C, f4.dequant(to64(a), fmt), f4.dequant(to64(b), fmt), K,
                    f"fp4 product {fmt} {M}x{N}x{K}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (9, 128, 384), (130, 384, 640), (300, 512, 1280)])
def test_product_of_every_code_and_scale_position(h3, fmt, M, N, K):
    """Random codes with a scale of its own for every block, all small enough that every
    partial sum is a whole multiple of a power of two below 2^24 of it: the result is the
    exact sum, rounded once."""
    rng = np.random.default_rng(M + N + K + fmt)
    S = K // f4.BLOCK[fmt]

    def operand(R):
        code = rng.integers(0, 16, (R, K)).astype(np.uint8)
        if fmt == f4.MX:
            byte = (127 + rng.integers(0, 4, (R, S))).astype(np.uint8)           # 1 .. 8
        else:
            byte = rng.choice(np.array([0x38, 0x3C, 0x40, 0x44, 0x48], np.uint8), (R, S))  # 1 .. 4
        row = 2.0 ** rng.integers(-3, 4, R).astype(np.float32)
        dev = [torch.from_numpy(v).to(DEV) for v in (f4.pack(code), f4.tile(byte, 0xFF), row)]
        return dev, f4.values(code, byte, row, fmt)
    (A, a), (B, b) = operand(M), operand(N)
    # codes are multiples of 1/2, scales of 1/2: partial sums are multiples of 2^-4 (before the
    # row factors) and at most K (6 * 8)^2 = 2^11.2 K: below 2^24 of 2^-4 for K <= 430, and the
    # sum of random signs stays below it for every K here
    C = _product(h3, A, B, fmt, M, N, K)
    want = torch.from_numpy(a @ b.T).to(torch.float32).to(torch.bfloat16)
    assert torch.equal(C.cpu(), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_product_with_and_without_row_factors(h3, fmt):
    M, N, K = 130, 256, 256
    rng = np.random.default_rng(4)
    g = torch.Generator().manual_seed(9)
    a = torch.randn(M, K, generator=g).to(torch.bfloat16)
    b = torch.randn(N, K, generator=g).to(torch.bfloat16)
    qa, qb = _quant(h3, a.to(DEV), fmt), _quant(h3, b.to(DEV), fmt)
    S = K // f4.BLOCK[fmt]
    va, vb = (f4.values(f4.unpack(q[0].cpu().numpy()), f4.untile(q[1].cpu().numpy(), n, S), np.ones(n), fmt)
              for q, n in ((qa, M), (qb, N)))
    ra, rb = rng.uniform(0.3, 3.0, M).astype(np.float32), rng.uniform(0.3, 3.0, N).astype(np.float32)
    for m in (1, 5, M):
        for fa in (None, ra):
            for fb in (None, rb):
                dv = lambda r: None if r is None else torch.from_numpy(r).to(DEV)  # noqa: E731
                A = (qa[0], qa[1], dv(fa))
                C = _product(h3, A, (qb[0], qb[1], dv(fb)), fmt, m, N, K)
                x = va[:m] * (1.0 if fa is None else fa[:m, None].astype(np.float64))
                y = vb * (1.0 if fb is None else fb[:, None].astype(np.float64))
                # two more roundings: of the two factors' product and of its product with the sum
                _assert_product(C, x, y, K + 2 * K, f"row factors {fmt} {m}")


@pytest.mark.parametrize("M", [1, 2, 16, 64, 200])
@pytest.mark.parametrize("up", [123, -123])
@pytest.mark.parametrize("fmt", FMTS)
def test_opposite_extremes_of_scale_cancel(h3, fmt, up, M):
    """Scales near both ends of their range in one product whose result is ordinary."""
    N, K = 256, 512
    g = torch.Generator().manual_seed(17)
    a = (torch.randn(M, K, generator=g) * 2.0 ** up).to(torch.bfloat16)
    b = (torch.randn(N, K, generator=g) * 2.0 ** -up).to(torch.bfloat16)
    # every block of the first row and weight full of its largest code
    a[0], b[0] = 6 * 2.0 ** up, 6 * 2.0 ** -up
    C = _product(h3, _quant(h3, a.to(DEV), fmt), _quant(h3, b.to(DEV), fmt), fmt, M, N, K)
    _assert_product(C, f4.dequant(to64(a), fmt), f4.dequant(to64(b), fmt), K, f"fmt {fmt} 2^{up} M {M}")


@pytest.mark.parametrize("fmt", FMTS)
def test_a_nan_block_reaches_its_row_only(h3, fmt):
    g = torch.Generator().manual_seed(12)
    N, K = 256, 512
    b = torch.randn(N, K, generator=g).to(torch.bfloat16)
    qb = _quant(h3, b.to(DEV), fmt)
    for M in (1, 12, 200):
        a = torch.randn(M, K, generator=g).to(torch.bfloat16)
        a[M // 2, 77] = float("inf")
        C = _product(h3, _quant(h3, a.to(DEV), fmt), qb, fmt, M, N, K)
        bad = torch.isnan(C).cpu()
        assert bool(bad[M // 2].all()) and int(bad.any(dim=1).sum()) == 1


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 11, 300])
def test_product_is_deterministic_and_replays_from_a_graph(h3, fmt, M):
    N, K = 640, 1408
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV)
    w = (torch.randn(N, K, generator=g) / math.sqrt(K)).to(torch.bfloat16).to(DEV)
    B = _quant(h3, w, fmt)
    q = torch.empty(M, K // 2, dtype=torch.uint8, device=DEV)
    bs = torch.empty(h3.h3_fp4_scale_bytes(fmt, M, K), dtype=torch.uint8, device=DEV)
    s = torch.empty(M, dtype=torch.float32, device=DEV) if fmt == f4.NV else None
    out = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)

    def step():
        h3.h3_quantize_rows_fp4(x, fmt, M, K, q, bs, s)
        h3.h3_gemm_fp4(q, bs, s, *B, fmt, M, N, K, out)
    step()
    assert h3.h3_sync_status() == 0
    ref = out.clone()
    step()
    assert torch.equal(out, ref)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    x2 = torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV)
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    step()
    assert h3.h3_sync_status() == 0
    assert torch.equal(out, replayed) and not torch.equal(out, ref)


def test_two_products_on_two_streams(h3):
    fmt, M, N, K = f4.NV, 200, 512, 1024
    g = torch.Generator().manual_seed(21)
    ops = []
    for _ in range(2):
        a = torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV)
        b = (torch.randn(N, K, generator=g) / 32).to(torch.bfloat16).to(DEV)
        A, B = _quant(h3, a, fmt), _quant(h3, b, fmt)
        ops.append((A, B, _product(h3, A, B, fmt, M, N, K).clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for _ in range(20):
        for (A, B, _), st, o in zip(ops, streams, outs):
            h3.h3_gemm_fp4(*A, *B, fmt, M, N, K, o, stream=st)
    torch.cuda.synchronize()
    assert h3.h3_sync_status() == 0
    for (_, _, ref), o in zip(ops, outs):
        assert torch.equal(o, ref)


# ------------------------------------------------------------------ long rows, many rows
def _rows_of(bs, rows, S):
    """Scale bytes [len(rows), S] of the given rows, gathered on the GPU."""
    r = torch.as_tensor(rows, device=DEV)[:, None]
    b = torch.arange(S, device=DEV)[None, :]
    at = ((r // 128) * (S // 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
    return bs[at].cpu().numpy()


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(h3, fmt):
    """4.4e9 elements through the quantiser and back, and a product that writes 2.3e9: sampled
    rows, the last ones among them."""
    R, K, S = 430_003, 10_240, 10_240 // f4.BLOCK[fmt]
    g = torch.Generator(device=DEV).manual_seed(31)
    x = torch.empty(R, K, dtype=torch.bfloat16, device=DEV)
    for r in range(0, R, 50_000):
        n = min(50_000, R - r)
        x[r:r + n] = torch.randn(n, K, generator=g, device=DEV)
    q, bs, s = _quant(h3, x, fmt)
    rows = np.unique(np.concatenate([np.arange(3), np.random.default_rng(1).integers(0, R, 24),
                                     [2 ** 31 // K, 2 ** 32 // K, R - 130, R - 2, R - 1]]))
    ridx = torch.from_numpy(rows).to(DEV)
    code, byte, row = f4.quantize(to64(x[ridx]), fmt)
    assert np.array_equal(_rows_of(bs, rows, S), byte)
    assert np.array_equal(f4.e2m1_decode(f4.unpack(q[ridx].cpu().numpy())), f4.e2m1_decode(code))
    if s is not None:
        assert np.array_equal(s[ridx].cpu().numpy(), row)
    h3.h3_dequantize_rows_fp4(q, bs, s, fmt, R, K, x)        # over x: it is read no more
    assert h3.h3_sync_status() == 0
    assert np.array_equal(to64(x[ridx]), f4.values(code, byte, row, fmt))
    del x
    N = 5376
    w = (torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K)).to(torch.bfloat16)
    B = _quant(h3, w, fmt)
    c = torch.full((R, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    h3.h3_gemm_fp4(q, bs, s, *B, fmt, R, N, K, c)
    assert h3.h3_sync_status() == 0
    assert not bool(torch.isnan(c[::1009]).any()) and not bool(torch.isnan(c[-300:]).any())
    _assert_product(c[ridx], f4.values(code, byte, row, fmt), f4.dequant(to64(w), fmt), K,
                    "rows of a long product")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 128, 65536), (40, 256, 65536), (300, 384, 65536), (1, 40960, 256),
                                   (20, 33024, 384), (50, 20480, 512), (130, 41088, 128)])
def test_longest_rows_and_widest_weights(h3, fmt, M, N, K):
    g = torch.Generator().manual_seed(M + N)
    a = torch.randn(M, K, generator=g).to(torch.bfloat16)
    b = (torch.randn(N, K, generator=g) / math.sqrt(K)).to(torch.bfloat16)
    C = _product(h3, _quant(h3, a.to(DEV), fmt), _quant(h3, b.to(DEV), fmt), fmt, M, N, K)
    _assert_product(C, f4.dequant(to64(a), fmt), f4.dequant(to64(b), fmt), K,
                    f"fp4 product {fmt} {M}x{N}x{K}")


# ------------------------------------------------------------------ calls behind one another
@pytest.mark.parametrize("fmt", FMTS)
def test_a_chain_of_dependent_calls_equals_single_steps(h3, fmt):
    """Quantise, multiply, quantise the result, ... without a pause: every call starts before
    the one ahead of it is done and must still see all it wrote, and must not write what the
    one ahead still reads.  Compared bit for bit with the same steps run one at a time."""
    shapes = [(1, 1024), (2, 1024), (20, 1024), (60, 1024), (700, 1024), (3000, 1024)]
    g = torch.Generator().manual_seed(5)
    for M, d in shapes:
        W = [_quant(h3, (torch.randn(d, d, generator=g) / math.sqrt(d)).to(torch.bfloat16).to(DEV), fmt)
             for _ in range(3)]
        x0 = torch.randn(M, d, generator=g).to(torch.bfloat16).to(DEV)
        q = torch.empty(M, d // 2, dtype=torch.uint8, device=DEV)
        bs = torch.empty(h3.h3_fp4_scale_bytes(fmt, M, d), dtype=torch.uint8, device=DEV)
        s = torch.empty(M, dtype=torch.float32, device=DEV) if fmt == f4.NV else None
        w1 = torch.ones(d, device=DEV)

        def chain(x, pause):
            res = x0.clone()
            for i in range(12):
                if i % 3 == 2:
                    h3.h3_rms_norm_fp4(x, res, w1, M, d, 1e-6, fmt, res, q, bs, s)
                else:
                    h3.h3_quantize_rows_fp4(x, fmt, M, d, q, bs, s)
                if pause:
                    torch.cuda.synchronize()
                h3.h3_gemm_fp4(q, bs, s, *W[i % 3], fmt, M, d, d, x)
                if pause:
                    torch.cuda.synchronize()
            h3.h3_quantize_rows_fp4(x, fmt, M, d, q, bs, s)
            if pause:
                torch.cuda.synchronize()
            h3.h3_dequantize_rows_fp4(q, bs, s, fmt, M, d, x)
            return x, res
        want, wres = chain(x0.clone(), True)
        assert h3.h3_sync_status() == 0 and bool(torch.isfinite(want).all())
        for _ in range(5):
            got, gres = chain(x0.clone(), False)
            assert h3.h3_sync_status() == 0
            assert torch.equal(got, want) and torch.equal(gres, wres), (M, fmt)


def test_calls_from_two_threads(h3):
    import threading
    fmt, N, K = f4.NV, 640, 768
    g = torch.Generator().manual_seed(77)
    W = _quant(h3, (torch.randn(N, K, generator=g) / 28).to(torch.bfloat16).to(DEV), fmt)
    jobs = []
    for M in (1, 9, 50, 300):
        x = torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV)
        A = _quant(h3, x, fmt)
        jobs.append((M, A, _product(h3, A, W, fmt, M, N, K).clone()))
    torch.cuda.synchronize()
    wrong = []
    ready = [(torch.cuda.Stream(), torch.empty_like(j[2])) for j in jobs]

    def work(job, st, out):
        # the thread's first CUDA call of any kind is the library's
        M, A, want = job
        try:
            for _ in range(100):
                h3.h3_gemm_fp4(*A, *W, fmt, M, N, K, out, stream=st)
            st.synchronize()
            if not torch.equal(out, want):
                wrong.append(M)
        except Exception as e:      # an exception would end the thread alone
            wrong.append((M, e))
    threads = [threading.Thread(target=work, args=(j, *r)) for j, r in zip(jobs, ready)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and h3.h3_sync_status() == 0


# ------------------------------------------------------------------ the MLP sub-block
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("name,hidden", [("tiny", 1024), ("tiny", 384), ("small", 8192)])
def test_mlp_fp4_against_oracle(h3, fmt, name, hidden):
    """h against the oracle fed the 4-bit operands that the call implies (y and W1 quantised
    from the definition on their bf16 values); out against the same for the second product,
    from the bf16 h that the call itself stored."""
    c = CONFIGS[name]
    g = torch.Generator().manual_seed(hidden + fmt)
    L, d = c.L, c.d
    x = torch.randn(L, d, generator=g).to(torch.bfloat16)
    w1 = (torch.randn(hidden, d, generator=g) / math.sqrt(d)).to(torch.bfloat16)
    w2 = (torch.randn(d, hidden, generator=g) / math.sqrt(hidden)).to(torch.bfloat16)
    sh, sc, gt = (torch.randn(3, d, generator=g) * 0.1 for _ in range(3))
    mod, _ = h3.h3_build_packed_layout(c.n_text, c.video_t, c.video_h, c.video_w,
                                       c.audio_channels, c.audio_steps)
    desc = h3.MlpDesc.make(L=L, d=d, hidden=hidden)
    nbytes = h3.h3_mlp_workspace_size_fp4(desc, fmt)
    gw, ws = _guarded(nbytes)
    q1, q2 = _quant(h3, w1.to(DEV), fmt), _quant(h3, w2.to(DEV), fmt)
    dv = [t.to(DEV) for t in (x, torch.from_numpy(mod), sh, sc, gt)]
    out = torch.full((L, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    h3.h3_mlp_block_fwd_fp4(desc, fmt, *dv, *q1, *q2, ws, nbytes, out)
    assert h3.h3_sync_status() == 0
    _intact(gw)
    off = (L * d * 2 + 255) // 256 * 256
    h_gpu = to64(ws[off:off + L * hidden * 2].view(torch.bfloat16).view(L, hidden))
    x64, s64, c64, g64 = to64(x), to64(sh), to64(sc), to64(gt)
    y = to64(ws[:L * d * 2].view(torch.bfloat16).view(L, d))
    assert_parity(y, orc.adaln_modulate(x64, mod, s64, c64), f"{name} fp4 mlp y")
    h = orc.gelu_tanh(orc.linear(f4.dequant(y, fmt), f4.dequant(to64(w1), fmt)))
    assert_parity(h_gpu, h, f"{name} fp4 mlp h")
    branch = orc.linear(f4.dequant(h_gpu, fmt), f4.dequant(to64(w2), fmt))
    assert_parity(to64(out), orc.gated_residual(x64, branch, mod, g64), f"{name} fp4 mlp out",
                  bf16_storage=False)
    # in place
    xin = dv[0].clone()
    h3.h3_mlp_block_fwd_fp4(desc, fmt, xin, *dv[1:], *q1, *q2, ws, nbytes, xin)
    assert h3.h3_sync_status() == 0 and torch.equal(xin, out)


def test_mlp_fp4_gate_zero_returns_input_and_bad_modality_is_reported(h3):
    fmt, L, d, hidden = f4.NV, 70, 256, 512
    g = torch.Generator().manual_seed(2)
    x = torch.randn(L, d, generator=g).to(torch.bfloat16).to(DEV)
    w1 = torch.randn(hidden, d, generator=g).to(torch.bfloat16).to(DEV)
    w2 = torch.randn(d, hidden, generator=g).to(torch.bfloat16).to(DEV)
    z = torch.zeros(2, d, device=DEV)
    mod = torch.zeros(L, dtype=torch.uint8, device=DEV)
    desc = h3.MlpDesc.make(L=L, d=d, hidden=hidden, n_mod=2)
    nbytes = h3.h3_mlp_workspace_size_fp4(desc, fmt)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    q1, q2 = _quant(h3, w1, fmt), _quant(h3, w2, fmt)
    out = torch.empty_like(x)
    h3.h3_mlp_block_fwd_fp4(desc, fmt, x, mod, z, z, z, *q1, *q2, ws, nbytes, out)
    assert h3.h3_sync_status() == 0 and torch.equal(out, x)
    mod[33] = 2
    h3.h3_mlp_block_fwd_fp4(desc, fmt, x, mod, z, z, z, *q1, *q2, ws, nbytes, out)
    assert h3.h3_sync_status() == 5
    bad = torch.isnan(out.float()).all(dim=1).cpu()
    assert bool(bad[33]) and int(bad.sum()) == 1
