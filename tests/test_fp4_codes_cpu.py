"""The test-side 4-bit quantiser against what its definition says, without a GPU."""
import numpy as np
import pytest

from tests._fp4 import (BLOCK, GRID, MX, NV, dequant, e2m1_decode, e2m1_round, half_step, pack,
                        quantize, scale_index, scale_values, scales, tile, unpack, untile)


def test_e2m1_rounds_to_nearest_even():
    for i in range(7):
        lo, hi = GRID[i], GRID[i + 1]
        mid = (lo + hi) / 2
        assert e2m1_round(mid) == (i if i % 2 == 0 else i + 1)
        assert e2m1_round(np.nextafter(mid, 0)) == i
        assert e2m1_round(np.nextafter(mid, 9)) == i + 1
        assert e2m1_round(-lo) & 7 == i and e2m1_round(hi) == i + 1
    assert e2m1_round(1e9) == 7 and e2m1_round(-7.0) == 15
    assert np.array_equal(e2m1_round(e2m1_decode(np.arange(16))), np.arange(16))


@pytest.mark.parametrize("fmt", [MX, NV])
def test_values_lie_within_half_a_step(fmt):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 384)) * 2.0 ** rng.integers(-20, 20, (40, 1))
    code, byte, row = quantize(x, fmt)
    s = (scale_values(byte, fmt) * row[:, None]).repeat(BLOCK[fmt], axis=1)
    t = x / np.where(s > 0, s, 1.0)
    if fmt == MX:
        assert np.all(np.abs(t) <= 6.0)                 # nothing is clipped
        a = np.abs(x).reshape(40, -1, 32).max(axis=2)
        assert np.all(a > 3.0 * scale_values(byte, fmt))  # and no smaller power would do
    t = np.clip(t, -6.0, 6.0)
    assert np.all(np.abs(e2m1_decode(code) - t)[s > 0] <= half_step(t)[s > 0])


def test_row_factor_uses_the_whole_scale_range():
    x = np.zeros((4, 128))
    x[0, 3], x[1, 7], x[2, 9] = 2688.0, 2689.0, 2.0 ** -130
    byte, row = scales(x, NV)
    assert row.tolist() == [1.0, 2.0, 2.0 ** -117, 1.0]
    assert scale_values(byte, NV)[0, 0] == 448.0 and scale_values(byte, NV)[1, 0] == 224.0
    assert np.all(dequant(x, NV)[3] == 0.0)


def test_packing_and_tiles_are_inverted():
    rng = np.random.default_rng(6)
    code = rng.integers(0, 16, (5, 128)).astype(np.uint8)
    assert np.array_equal(unpack(pack(code)), code) and pack(code)[0, 0] & 15 == code[0, 0]
    for R, S in ((1, 4), (130, 8), (257, 12)):
        b = rng.integers(0, 255, (R, S)).astype(np.uint8)
        flat = tile(b)
        assert flat.size == (R + 127) // 128 * 128 * S
        assert len(np.unique(scale_index(R, S))) == R * S
        assert np.array_equal(untile(flat, R, S), b)
    # 128 rows x 4 blocks a tile; row r at 16 (r % 32) + 4 (r // 32)
    i = scale_index(256, 8)
    assert i[0, 0] == 0 and i[1, 0] == 16 and i[32, 0] == 4 and i[0, 4] == 512 and i[128, 0] == 1024
