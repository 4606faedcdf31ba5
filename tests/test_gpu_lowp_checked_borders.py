"""The checked build's tests of extents at the borders of the 4-bit and norm kernels: the last
row of a 128-row group and the first of the next, widths that leave part of a warp's step, every
number of warps a row, rows that are summed again, the row counts where product kernels change.
Nothing reported, and the same bits as the library."""
import math

import pytest
import torch

import joint_audio_video_gb300 as h3lib
from tests.test_gpu_checked import _both, checked  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"
MX, NV = 1, 2


def _room(fmt, R, K):
    return (torch.zeros(R, K // 2, dtype=torch.uint8, device=DEV),
            torch.zeros(h3lib.h3_fp4_scale_bytes(fmt, R, K), dtype=torch.uint8, device=DEV),
            torch.ones(R, device=DEV))


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("R,K", [(1, 128), (127, 384), (128, 2048), (129, 5120), (300, 1152), (33, 8320),
                                 (5, 20480), (3, 65536)])
def test_quantiser_and_inverse(h3, checked, fmt, R, K):  # noqa: F811
    x = torch.randn(R, K, generator=torch.Generator().manual_seed(R)).to(torch.bfloat16).to(DEV)

    def run():
        q, bs, s = _room(fmt, R, K)
        h3lib.h3_quantize_rows_fp4(x, fmt, R, K, q, bs, s)
        y = torch.empty_like(x)
        h3lib.h3_dequantize_rows_fp4(q, bs, s, fmt, R, K, y)
        return q, bs, s, y
    _both(checked, run)


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("L,d", [(1, 128), (129, 256), (6, 384), (7, 512), (9, 640), (130, 1152), (127, 2048),
                                 (128, 5120), (5, 16384)])
def test_norms(h3, checked, L, d, eps):  # noqa: F811
    g = torch.Generator().manual_seed(L + d)
    x = torch.randn(L, d, generator=g)
    x *= torch.exp2(torch.tensor([0.0, 120.0, 66.0, -70.0])[torch.arange(L) % 4])[:, None]
    x, res = x.to(torch.bfloat16).to(DEV), torch.randn(L, d, generator=g).to(torch.bfloat16).to(DEV)
    w = torch.rand(d, generator=g).to(DEV)

    def run():
        out = []
        for r in (res, None):
            q, sc, s = torch.empty(L, d, dtype=torch.uint8, device=DEV), torch.empty(L, device=DEV), torch.empty_like(x)
            h3lib.h3_rms_norm_fp8(x, r, w, L, d, eps, s, q, sc)
            out += [q, sc, s]
            for fmt in (MX, NV):
                o = _room(fmt, L, d)
                h3lib.h3_rms_norm_fp4(x, r, w, L, d, eps, fmt, None, *o)
                out += o
        return out
    _both(checked, run)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (1, 5120, 640), (2, 384, 4096), (3, 256, 8192), (16, 128, 65536),
                                   (17, 640, 384), (48, 256, 1152), (64, 128, 8192), (65, 192 * 2, 256),
                                   (129, 256, 640), (257, 640, 384)])
def test_products(h3, checked, fmt, M, N, K):  # noqa: F811
    g = torch.Generator().manual_seed(M + N)
    a = torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV)
    b = (torch.randn(N, K, generator=g) / math.sqrt(K)).to(torch.bfloat16).to(DEV)
    far = torch.full((M,), 2.0 ** 70, device=DEV)

    def run():
        A, B = _room(fmt, M, K), _room(fmt, N, K)
        h3lib.h3_quantize_rows_fp4(a, fmt, M, K, *A)
        h3lib.h3_quantize_rows_fp4(b, fmt, N, K, *B)
        out = []
        for fa, fb in ((None, None), (A[2], B[2]), (far, B[2])):
            c = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
            h3lib.h3_gemm_fp4(A[0], A[1], fa, B[0], B[1], fb, fmt, M, N, K, c)
            out.append(c)
        return out
    _both(checked, run)
