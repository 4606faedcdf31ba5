"""h3_gemm_fp8 with scales near the ends of fp32's range: right whenever the result is in range,
although a_scale x b_scale is not.

Bound: the bf16 rounding of the result (2^-8 of it, at least 2^-134), one rounding of at most
2^-23 of sum |a b| for each of K products and K / 32 steps, and 2^-23 each for the scales'
product, its product with the sum and a step that ends below the normal numbers."""
import numpy as np
import pytest
import torch

from tests._fp8 import e4m3_decode
from tests._parity import to64
from tests.test_gpu_fp8 import _quant
from tests.test_gpu_row_factors import LARGEST, _factors
from tests.test_gpu_fp4 import to64_nan

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _check(C, a, b, sa, sb, what):
    K = a.shape[1]
    f = sa.astype(np.float64)[:, None] * sb.astype(np.float64)[None, :]
    ref, mag = (a @ b.T) * f, (np.abs(a) @ np.abs(b).T) * np.abs(f)
    got = to64_nan(C)
    tol = 2.0 ** -8 * np.abs(ref) + (K + K // 32 + 3) * 2.0 ** -23 * mag + 2.0 ** -134
    beyond, near = np.abs(ref) - tol >= LARGEST, np.abs(ref) + tol >= LARGEST
    assert np.array_equal(got[beyond], np.copysign(np.inf, ref[beyond])), what
    with np.errstate(invalid="ignore"):
        wrong = ~(np.abs(got - ref) <= tol) & ~near
    assert not wrong.any(), (what, int(wrong.sum()), got[wrong][:4], ref[wrong][:4])


# 700 rows and 1,024 columns: pairs of CTAs; the others: one CTA a tile
@pytest.mark.parametrize("M,N,K", [(1, 128, 256), (200, 384, 640), (700, 1024, 512)])
@pytest.mark.parametrize("ea,eb", [(-80, -70), (70, 60), (64, 64), (126, -140), (-149, 100), (0, 0)])
def test_fp8_product_under_extreme_scales(h3, M, N, K, ea, eb):
    rng = np.random.default_rng(1000 + M + ea)
    codes = np.arange(256, dtype=np.uint8)
    codes = codes[(codes & 0x7F) != 0x7F]
    A, B = rng.choice(codes, (M, K)), rng.choice(codes, (N, K))
    A[M // 2], B[N // 2] = 0, 0
    sa, sb = _factors(rng, M, ea), _factors(rng, N, eb)
    dv = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    h3.h3_gemm_fp8(dv(A), dv(sa), dv(B), dv(sb), M, N, K, C)
    assert h3.h3_sync_status() == 0
    _check(C, e4m3_decode(A), e4m3_decode(B), sa, sb, f"{M}x{N}x{K} 2^{ea} 2^{eb}")


@pytest.mark.parametrize("M", [1, 200])
@pytest.mark.parametrize("e", [-66, 75])
def test_fp8_product_of_two_small_or_two_large_matrices(h3, M, e):
    """The large ones meet in no column: their product is zero."""
    N, K = 256, 4096
    g = torch.Generator().manual_seed(5)
    a = (torch.rand(M, K, generator=g) + 0.5) * 2.0 ** e
    b = (torch.rand(N, K, generator=g) + 0.5) * 2.0 ** e
    if e > 0:
        a[:, : K // 2], b[:, K // 2:] = 0.0, 0.0
    (qa, sa), (qb, sb) = _quant(h3, a.to(torch.bfloat16).to(DEV)), _quant(h3, b.to(torch.bfloat16).to(DEV))
    C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    h3.h3_gemm_fp8(qa, sa, qb, sb, M, N, K, C)
    assert h3.h3_sync_status() == 0
    _check(C, e4m3_decode(qa.cpu().numpy()), e4m3_decode(qb.cpu().numpy()), sa.cpu().numpy(),
           sb.cpu().numpy(), f"2^{e} M {M}")
    assert bool((C == 0).all()) == (e > 0)
    assert e > 0 or float(to64(C).min()) > 2.0 ** -126
