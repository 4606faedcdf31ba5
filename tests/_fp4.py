"""Microscaled 4-bit matrices from their definition, in float64 (test helper, no method
arithmetic): E2M1 codes (0 .5 1 1.5 2 3 4 6 and a sign), an E8M0 scale for 32 columns (MX)
or an E4M3 scale for 16 columns and a power of two for each row (NV)."""
import numpy as np

from tests._fp8 import e4m3_decode, e4m3_round

MX, NV = 1, 2
BLOCK = {MX: 32, NV: 16}
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_round(t):
    """E2M1 code of each value: to nearest, ties to the even code, 6 at most."""
    t = np.asarray(t, dtype=np.float64)
    a = np.minimum(np.abs(t), 6.0)
    hi = np.clip(np.searchsorted(GRID, a), 1, 7)
    lo = hi - 1
    up, down = GRID[hi] - a, a - GRID[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(lo % 2 == 0, lo, hi)))
    return (code | (np.signbit(t).astype(np.int64) << 3)).astype(np.uint8)


def e2m1_decode(c):
    c = np.asarray(c)
    return np.where(c & 8, -1.0, 1.0) * GRID[c & 7]


def half_step(t):
    """Half the distance between the E2M1 values around |t| <= 6."""
    a = np.abs(t)
    return np.where(a < 2.0, 0.25, np.where(a < 4.0, 0.5, 1.0))


def _smallest_power(x, most):
    """k = min{k : x <= most * 2^k} for x > 0."""
    k = np.ceil(np.log2(x / most))
    k = np.where(most * 2.0 ** (k - 1) >= x, k - 1, k)
    return np.where(most * 2.0 ** k < x, k + 1, k)


def scales(x, fmt):
    """(scale bytes [R, S], row factors [R]) of ``x [R, K]`` (finite)."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    a = np.abs(x).reshape(R, K // BLOCK[fmt], BLOCK[fmt]).max(axis=2)
    if fmt == MX:
        k = np.where(a > 0, np.maximum(_smallest_power(np.where(a > 0, a, 1.0), 6.0), -127), -127)
        return (k + 127).astype(np.uint8), np.ones(R)
    top = a.max(axis=1)
    e = np.where(top > 0, np.maximum(_smallest_power(np.where(top > 0, top, 1.0), 2688.0), -117), 0)
    row = 2.0 ** e
    return e4m3_round(a / row[:, None] / 6.0), row


def scale_values(byte, fmt):
    if fmt == MX:
        return np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127.0))
    return np.where((byte & 0x7F) == 0x7F, np.nan, e4m3_decode(byte))


def quantize(x, fmt):
    """(codes [R, K], scale bytes [R, S], row factors [R])."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    byte, row = scales(x, fmt)
    s = scale_values(byte, fmt) * row[:, None]
    b = x.reshape(R, -1, BLOCK[fmt])
    live = (s > 0)[:, :, None]
    t = np.where(live, b / np.where(live, s[:, :, None], 1.0), 0.0)
    return e2m1_round(t).reshape(R, K), byte, row


def values(code, byte, row, fmt):
    R, K = code.shape
    s = scale_values(byte, fmt) * np.asarray(row, dtype=np.float64)[:, None]
    return (e2m1_decode(code).reshape(R, -1, BLOCK[fmt]) * s[:, :, None]).reshape(R, K)


def dequant(x, fmt):
    return values(*quantize(x, fmt), fmt)


def pack(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    out = np.empty((q.shape[0], 2 * q.shape[1]), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def scale_index(R, S):
    """Byte of block b of row r in the tiled scale array: [R, S]."""
    r, b = np.arange(R)[:, None], np.arange(S)[None, :]
    return ((r // 128) * (S // 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4


def tile(byte, fill=0):
    R, S = byte.shape
    out = np.full((R + 127) // 128 * 128 * S, fill, dtype=np.uint8)
    out[scale_index(R, S)] = byte
    return out


def untile(flat, R, S):
    return np.asarray(flat)[scale_index(R, S)]
