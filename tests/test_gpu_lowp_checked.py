"""The 4-bit products and the quantising norms through the checked build (every global access
that a kernel addresses itself tested against its buffer): nothing reported, the same bits."""
import math

import pytest
import torch

import joint_audio_video_gb300 as h3lib
from tests._fp4 import MX, NV
from tests.test_gpu_checked import _both, checked  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("M", [1, 2, 30, 61, 130, 700])
def test_checked_products_and_norms_match(h3, checked, fmt, M):  # noqa: F811
    N, K = 640, 1152
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV)
    res = torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV)
    w = (torch.randn(N, K, generator=g) / math.sqrt(K)).to(torch.bfloat16).to(DEV)
    wt = torch.ones(K, device=DEV)

    def run():
        out = []
        room = []
        for R in (M, N):
            n = h3lib.h3_fp4_scale_bytes(fmt, R, K)
            room.append((torch.empty(R, K // 2, dtype=torch.uint8, device=DEV),
                         torch.zeros(n, dtype=torch.uint8, device=DEV),
                         torch.ones(R, device=DEV)))
        (q, bs, s), B = room
        h3lib.h3_quantize_rows_fp4(w, fmt, N, K, *B)
        h3lib.h3_quantize_rows_fp4(x, fmt, M, K, q, bs, s)
        y = torch.empty_like(x)
        h3lib.h3_dequantize_rows_fp4(q, bs, s, fmt, M, K, y)
        C = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        h3lib.h3_gemm_fp4(q, bs, s, *B, fmt, M, N, K, C)
        out += [q.clone(), bs.clone(), s.clone(), y, C.clone()]
        r = res.clone()
        h3lib.h3_rms_norm_fp4(x, r, wt, M, K, 1e-6, fmt, r, q, bs, s)
        h3lib.h3_gemm_fp4(q, bs, s, *B, fmt, M, N, K, C)
        q8, s8 = torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(M, device=DEV)
        h3lib.h3_rms_norm_fp8(x, r, wt, M, K, 1e-6, None, q8, s8)
        return out + [q, bs, s, C, r, q8, s8]

    _both(checked, run)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("L", [1, 40, 300])
def test_checked_mlp_matches(h3, checked, fmt, L):  # noqa: F811
    d, hidden = 256, 640
    g = torch.Generator().manual_seed(L)
    x = torch.randn(L, d, generator=g).to(torch.bfloat16).to(DEV)
    sh, sc, gt = (0.1 * torch.randn(3, d, generator=g).to(DEV) for _ in range(3))
    mod = (torch.arange(L) % 3).to(torch.uint8).to(DEV)
    ws = [(torch.randn(n, k, generator=g) / math.sqrt(k)).to(torch.bfloat16).to(DEV)
          for n, k in ((hidden, d), (d, hidden))]
    desc = h3lib.MlpDesc.make(L=L, d=d, hidden=hidden)

    def run():
        W = []
        for w in ws:
            R, K = w.shape
            W += [torch.empty(R, K // 2, dtype=torch.uint8, device=DEV),
                  torch.zeros(h3lib.h3_fp4_scale_bytes(fmt, R, K), dtype=torch.uint8, device=DEV),
                  torch.ones(R, device=DEV)]
            h3lib.h3_quantize_rows_fp4(w, fmt, R, K, *W[-3:])
        n = h3lib.h3_mlp_workspace_size_fp4(desc, fmt)
        work = torch.empty(n, dtype=torch.uint8, device=DEV)
        out = torch.empty_like(x)
        h3lib.h3_mlp_block_fwd_fp4(desc, fmt, x, mod, sh, sc, gt, *W, work, n, out)
        return (out,)

    _both(checked, run)
