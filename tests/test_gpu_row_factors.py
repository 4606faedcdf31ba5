"""Row factors near the ends of fp32's range: a product, or what a 4-bit matrix stands for, is
right whenever the value itself is in range, although the two factors' product is not.

Bound of a product: the bf16 rounding of the result (2^-8 of it, at least 2^-134, half of
bf16's smallest step), one rounding of at most 2^-23 of sum |a b| for each of K products and
K / 64 steps, and 2^-23 each for the factors' product, its product with the sum and a step
that ends below the normal numbers."""
import math

import numpy as np
import pytest
import torch

from tests import _fp4 as f4
from tests._parity import BF16_U, to64
from tests.test_gpu_fp4 import _quant, to64_nan

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMTS = [f4.MX, f4.NV]
LARGEST = 2.0 ** 127 * (2.0 - 2.0 ** -8)      # from here on bf16 rounds to infinity


def _check(C, a, b, ra, rb, what):
    """C against (a b^T) ra rb: a [M][K], b [N][K] without their row factors."""
    K = a.shape[1]
    f = ra.astype(np.float64)[:, None] * rb.astype(np.float64)[None, :]
    ref, mag = (a @ b.T) * f, (np.abs(a) @ np.abs(b).T) * np.abs(f)
    got = to64_nan(C)
    tol = BF16_U * np.abs(ref) + (K + K // 64 + 3) * 2.0 ** -23 * mag + 2.0 ** -134
    beyond, near = np.abs(ref) - tol >= LARGEST, np.abs(ref) + tol >= LARGEST
    assert np.array_equal(got[beyond], np.copysign(np.inf, ref[beyond])), what
    with np.errstate(invalid="ignore"):
        wrong = ~(np.abs(got - ref) <= tol) & ~near
    assert not wrong.any(), (what, int(wrong.sum()), got[wrong][:4], ref[wrong][:4])


def _operand(rng, R, K, fmt, scale_exp, zero_row=None, columns=None):
    """Random codes under power-of-two block scales around 2^scale_exp: (codes, scales) on the
    GPU, and the values without row factors."""
    S = K // f4.BLOCK[fmt]
    code = rng.integers(0, 16, (R, K)).astype(np.uint8)
    if zero_row is not None:
        code[zero_row] = 0
    if columns is not None:
        code[:, columns:] = 0
    e = scale_exp + rng.integers(0, 3, (R, S))
    byte = (e + 127).astype(np.uint8) if fmt == f4.MX else ((e + 7) << 3).astype(np.uint8)
    dv = [torch.from_numpy(v).to(DEV) for v in (f4.pack(code), f4.tile(byte, 0xFF))]
    return dv, f4.values(code, byte, np.ones(R), fmt)


def _factors(rng, n, e):
    """n factors of either sign with the exponents e, e - 1, 0 and 1 mixed."""
    pick = np.array([e, e - 1, e, 0, 1])[rng.integers(0, 5, n)]
    pick[0] = e
    return (rng.uniform(1.0, 2.0, n) * rng.choice([-1.0, 1.0], n) * 2.0 ** pick).astype(np.float32)


# M: one and two rows without tensor cores, few rows, pairs of CTAs
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 2, 13, 40, 200])
@pytest.mark.parametrize("ea,eb", [(-75, -75), (-74, -76), (70, 70), (64, 64), (126, -140), (-149, 100),
                                   (100, -60), (-126, 3)])
def test_product_under_extreme_row_factors(h3, fmt, M, ea, eb):
    N, K = 384, 640
    rng = np.random.default_rng(1000 * M + 7 * ea + eb)
    # sums that bring a small pair of factors back into range, and a large pair; MX scales reach
    # further than E4M3's, whose exponents end at -6 and 8
    up = -(ea + eb) // 2
    lim = 50 if fmt == f4.MX else 5
    up = max(-lim, min(lim, up))
    A, a = _operand(rng, M, K, fmt, up, zero_row=M // 2 if M > 2 else None)
    B, b = _operand(rng, N, K, fmt, up, zero_row=N // 2)
    for x, y, ex, ey in ((M, N, ea, eb), (M, N, eb, ea)):
        ra, rb = _factors(rng, x, ex), _factors(rng, y, ey)
        C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
        h3.h3_gemm_fp4(*A, torch.from_numpy(ra).to(DEV), *B, torch.from_numpy(rb).to(DEV), fmt, M, N,
                       K, C)
        assert h3.h3_sync_status() == 0
        _check(C, a, b, ra, rb, f"fmt {fmt} M {M} 2^{ex} 2^{ey}")


@pytest.mark.parametrize("M", [1, 2, 13, 40, 200])
@pytest.mark.parametrize("ea,eb", [(100, 33), (-20, 120), (70, 70)])
def test_sums_below_the_normal_numbers_under_large_factors(h3, M, ea, eb):
    """MX scales whose products are far below fp32's normal numbers: sums of three products are
    whole multiples of 2^-148, so exact, and the factors bring them back.  One or two rows hold
    sums to 2^-139: scales 2^10 larger."""
    N, K = 256, 128
    rng = np.random.default_rng(1000 + M + ea)
    up = -73 if M > 2 else -68
    A, a = _operand(rng, M, K, f4.MX, up, columns=3)
    B, b = _operand(rng, N, K, f4.MX, up)
    ra, rb = _factors(rng, M, ea), _factors(rng, N, eb)
    C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    h3.h3_gemm_fp4(*A, torch.from_numpy(ra).to(DEV), *B, torch.from_numpy(rb).to(DEV), f4.MX, M, N, K, C)
    assert h3.h3_sync_status() == 0
    _check(C, a, b, ra, rb, f"M {M} 2^{ea} 2^{eb}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 2, 13, 40, 200])
def test_zero_and_absent_row_factors(h3, fmt, M):
    N, K = 256, 256
    rng = np.random.default_rng(M)
    A, a = _operand(rng, M, K, fmt, 0)
    B, b = _operand(rng, N, K, fmt, 0)
    ra, rb = _factors(rng, M, 90), _factors(rng, N, 90)
    ra[M // 2], rb[3], rb[200] = 0.0, 0.0, -0.0
    one = lambda n: np.ones(n, dtype=np.float32)  # noqa: E731
    dv = lambda r: torch.from_numpy(r).to(DEV)  # noqa: E731
    for fa, fb in ((ra, rb), (ra, None), (None, rb)):
        C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
        h3.h3_gemm_fp4(*A, None if fa is None else dv(fa), *B, None if fb is None else dv(fb), fmt, M,
                       N, K, C)
        assert h3.h3_sync_status() == 0
        _check(C, a, b, one(M) if fa is None else fa, one(N) if fb is None else fb, f"fmt {fmt} M {M}")


@pytest.mark.parametrize("M", [1, 2, 16, 40, 200])
@pytest.mark.parametrize("e", [-66, -64, 40, 75])
@pytest.mark.parametrize("fmt", FMTS)
def test_product_of_two_small_or_two_large_matrices(h3, fmt, e, M):
    """Both operands quantised from values around 2^e.  The large ones meet in no column, so that
    their product is zero although their row factors' product may be infinite."""
    N, K = 256, 4096
    g = torch.Generator().manual_seed(5)
    a = (torch.rand(M, K, generator=g) + 0.5) * 2.0 ** e
    b = (torch.rand(N, K, generator=g) + 0.5) * 2.0 ** e
    if e > 0:
        a[:, : K // 2], b[:, K // 2:] = 0.0, 0.0
    a, b = a.to(torch.bfloat16), b.to(torch.bfloat16)
    A, B = _quant(h3, a.to(DEV), fmt), _quant(h3, b.to(DEV), fmt)
    C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    h3.h3_gemm_fp4(*A, *B, fmt, M, N, K, C)
    assert h3.h3_sync_status() == 0
    one = lambda n: np.ones(n, dtype=np.float32)  # noqa: E731
    va, vb = f4.dequant(to64(a), fmt), f4.dequant(to64(b), fmt)
    _check(C, va, vb, one(M), one(N), f"fmt {fmt} 2^{e} M {M}")
    if e > 0:
        assert bool((C == 0).all())
    else:
        assert math.log2(float(to64(C).min())) > -126
