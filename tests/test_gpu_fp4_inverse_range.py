"""h3_dequantize_rows_fp4 under any fp32 row factors: right wherever the value is in range,
whatever code x factor or factor x scale alone would be.

Bound: one rounding of code x scale x factor in fp32 and one where it ends below the normal
numbers (2^-24 of the value each, at least 2^-150), and the bf16 rounding (2^-8, at least
2^-134)."""
import numpy as np
import pytest
import torch

from tests import _fp4 as f4
from tests._parity import BF16_U
from tests.test_gpu_fp4 import to64_nan

pytestmark = pytest.mark.gpu
DEV = "cuda"
LARGEST = 2.0 ** 127 * (2.0 - 2.0 ** -8)      # from here on bf16 rounds to infinity


@pytest.mark.parametrize("fmt", [f4.MX, f4.NV])
@pytest.mark.parametrize("e", [127, 126, 100, 24, 0, -24, -100, -126, -133, -148])
def test_inverse_under_extreme_row_factors(h3, fmt, e):
    rng = np.random.default_rng(e + 1000)
    R, K = 140, 384
    S = K // f4.BLOCK[fmt]
    code = rng.integers(0, 16, (R, K)).astype(np.uint8)
    byte = rng.integers(0, 255 if fmt == f4.MX else 127, (R, S)).astype(np.uint8)
    # scales that bring the factor back to ordinary values, the smallest, one and two
    near = np.clip(127 - e + rng.integers(-3, 4, (R, S)), 0, 254).astype(np.uint8)
    if fmt == f4.MX:
        byte = np.where(rng.random((R, S)) < 0.6, near, byte)
        byte[:, :4] = [0, 1, 127, 128]
        byte[5, 6] = 255
    row = (rng.uniform(1.0, 2.0, R) * rng.choice([-1.0, 1.0], R) * 2.0 ** e).astype(np.float32)
    row[3] = np.float32(2.0 ** e)
    row[7] = 0.0
    dv = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    y = torch.empty(R, K, dtype=torch.bfloat16, device=DEV)
    h3.h3_dequantize_rows_fp4(dv(f4.pack(code)), dv(f4.tile(byte, 0x55)), dv(row), fmt, R, K, y)
    assert h3.h3_sync_status() == 0
    want = f4.values(code, byte, row, fmt)
    got = to64_nan(y)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    tol = (BF16_U + 2.0 ** -23) * np.abs(want) + 2.0 ** -134 + 2.0 ** -149
    with np.errstate(invalid="ignore"):
        beyond, near = np.abs(want) - tol >= LARGEST, np.abs(want) + tol >= LARGEST
        assert np.array_equal(got[beyond], np.copysign(np.inf, want[beyond]))
        ok = ~np.isnan(want) & ~near
        wrong = ok & ~(np.abs(got - want) <= tol)
    assert not wrong.any(), (fmt, e, int(wrong.sum()), got[wrong][:4], want[wrong][:4])


def test_a_large_factor_under_a_small_scale(h3):
    """Code 6, row factor 2^126, scale 2^-100: 6 x 2^26."""
    K = 128
    q = torch.full((1, K // 2), 0x77, dtype=torch.uint8, device=DEV)
    bs = torch.full((h3.h3_fp4_scale_bytes(f4.MX, 1, K),), 27, dtype=torch.uint8, device=DEV)
    y = torch.empty(1, K, dtype=torch.bfloat16, device=DEV)
    h3.h3_dequantize_rows_fp4(q, bs, torch.full((1,), 2.0 ** 126, device=DEV), f4.MX, 1, K, y)
    assert h3.h3_sync_status() == 0
    assert bool((y == 6 * 2.0 ** 26).all())
