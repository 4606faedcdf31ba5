"""Cases of the low-precision operators: microscaled 4-bit quantisation and
product, and the root-mean-square norm with the residual's addition whose
output is held in 8 or 4 bits.

Each case is one pass through one operator (or, for "norm_product", the two in
the order a layer calls them).  With ``own`` false, ``run`` computes the plain
form in elementary torch operations in 32 bits; with ``own`` true it calls the
library.  ``exact`` computes the same outputs from the definitions in 64 bits.

Formats of a 4-bit matrix [R][K] (two E2M1 codes a byte, the even column in the
low half), block scales in tiles of 128 rows x 4 scales (512 bytes; row r of
the tile at 16 (r % 32) + 4 (r // 32)):
  "mx"  one E8M0 (power of two) scale for 32 columns
  "nv"  one E4M3 scale for 16 columns, times one power of two for each row
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = {"mx": 32, "nv": 16}
EPS = 1e-6
# the largest product: the up projection of a full-size request
MOST = 58758 * 20480 * 5120


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token's activations on their way into a 4-bit projection: latency
        {"name": "quant_mx_one_token", "op": "quant", "fmt": "mx", "R": 1, "K": 5120},
        # all tokens of a full-size request, as before every projection of a layer
        {"name": "quant_nv_full", "op": "quant", "fmt": "nv", "R": 58758, "K": 5120},
        # output projection for one token: the weights' bytes and the launch
        {"name": "product_nv_one_token", "op": "product", "fmt": "nv", "M": 1, "N": 5120, "K": 5120},
        # the text tokens of a request through the feed-forward up projection: a ragged
        # row count, a few tiles
        {"name": "product_mx_text", "op": "product", "fmt": "mx", "M": 358, "N": 20480, "K": 5120},
        # QKV projection of the small workload
        {"name": "product_nv_small", "op": "product", "fmt": "nv", "M": 4096, "N": 6144, "K": 2048},
        # feed-forward down projection over an odd number of tokens: a long sum
        {"name": "product_mx_odd", "op": "product", "fmt": "mx", "M": 1501, "N": 2048, "K": 8192},
        # feed-forward up projection of a full-size request
        {"name": "product_nv_full", "op": "product", "fmt": "nv", "M": 58758, "N": 20480, "K": 5120},
        # the norm of one token: latency
        {"name": "norm_one_token", "op": "norm", "L": 1, "d": 5120},
        # an odd number of tokens of the small workload's width
        {"name": "norm_odd", "op": "norm", "L": 4099, "d": 2048},
        # all tokens of a full-size request
        {"name": "norm_full", "op": "norm", "L": 58758, "d": 5120},
        # a handful of tokens through a norm into their 4-bit QKV projection
        {"name": "norm_product_nv_few", "op": "norm_product", "fmt": "nv", "M": 13, "N": 15360, "K": 5120},
        # the small workload through a norm into its 4-bit up projection
        {"name": "norm_product_mx_small", "op": "norm_product", "fmt": "mx", "M": 4096, "N": 8192, "K": 2048},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log128(rng, hi):
    return 128 * min(hi // 128, max(1, _log(rng, 128, hi) // 128))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "norm", "norm_product"])
    fmt = rng.choice(["mx", "nv"])
    if op == "norm":
        return {"op": op, "L": _log(rng, 1, 58758), "d": _log128(rng, 8192)}
    if op == "quant":
        K = _log128(rng, 20480)
        return {"op": op, "fmt": fmt, "R": _log(rng, 1, min(58758, 58758 * 5120 // K)), "K": K}
    # the norm's width is at most 16,384
    N, K = _log128(rng, 20480), _log128(rng, 20480 if op == "product" else 8192)
    return {"op": op, "fmt": fmt, "M": _log(rng, 1, min(58758, MOST // (N * K))), "N": N, "K": K}


def work(case):
    c = case
    if c["op"] == "quant":
        # bf16 read, the bf16 values it stands for written
        return {"bytes": 4 * c["R"] * c["K"], "flops": 4 * c["R"] * c["K"]}
    if c["op"] == "norm":
        n = c["L"] * c["d"]
        return {"bytes": 7 * n + 4 * c["L"] + 4 * c["d"], "flops": 8 * n}
    M, N, K = c["M"], c["N"], c["K"]
    per = 0.5 + 1 / BLOCK[c["fmt"]]         # bytes of a 4-bit element with its scale
    flops = 2 * M * N * K
    if c["op"] == "product":
        return {"bytes": int((M + N) * K * per) + 2 * M * N, "flops": flops}
    return {"bytes": int(N * K * per) + 6 * M * K + 4 * K + 2 * M * N, "flops": flops + 8 * M * K}


# ------------------------------------------------------------------ plain form (32 bits)
def _pow2(e):
    """2^e in fp32 for an integer tensor e in [-126, 127]: the exponent field written out."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _times_pow2(x, e):
    """x 2^e for e in [-252, 254], in two factors that fp32 holds."""
    h = torch.div(e, 2, rounding_mode="floor")
    return x * _pow2(h) * _pow2(e - h)


def _exponent_and_mantissa(a):
    """a = m 2^e with 1 <= m < 2 (fp32; 0 gives m = 0)."""
    m, e = torch.frexp(a)
    return e - 1, 2 * m


def _e2m1_index(a):
    """Index 0..7 of the nearest of {0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the even index."""
    i = (a > 0.25).to(torch.uint8)
    i += a >= 0.75
    i += a > 1.25
    i += a >= 1.75
    i += a > 2.5
    i += a >= 3.5
    i += a > 5.0
    return i


def _quantize(x, fmt):
    """fp32 x [R][K] -> codes (uint8, one a value), block scales (fp32), row scales (fp32 or None)."""
    R, K = x.shape
    b = x.view(R, K // BLOCK[fmt], BLOCK[fmt])
    amax = b.abs().amax(2)
    if fmt == "mx":
        # the smallest power of two with amax / scale <= 6
        e, m = _exponent_and_mantissa(amax)
        k = torch.where(m <= 1.5, e - 2, e - 1).clamp(-127, 127)
        k = torch.where(amax > 0, k, torch.full_like(k, -127))
        scale, row = _times_pow2(torch.ones_like(amax), k), None
        v = _times_pow2(b, -k[:, :, None])
    else:
        # the smallest power of two with amax / (6 row) <= 448
        top = amax.amax(1)
        e, m = _exponent_and_mantissa(top)
        e = torch.where(m <= 1.3125, e - 11, e - 10).clamp(-126, 126)
        e = torch.where(top > 0, e, torch.zeros_like(e))
        row, inv = _pow2(e), _pow2(-e)
        # divided by a tensor: a number would be turned into a product with its rounded inverse
        scale = (amax * inv[:, None] / torch.full_like(amax, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
        s = scale[:, :, None]
        v = torch.where(s > 0, b * inv[:, None, None] / s, torch.zeros_like(b))
    code = _e2m1_index(v.abs()) + (torch.signbit(b).to(torch.uint8) << 3)
    return code.view(R, K), scale, row


def _pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _unpack(q):
    return torch.stack((q & 15, q >> 4), dim=2).flatten(1)


def _scale_bytes(scale, fmt):
    if fmt == "mx":
        return (torch.log2(scale.double()).round().to(torch.int32) + 127).to(torch.uint8)
    return scale.to(torch.float8_e4m3fn).view(torch.uint8)


def _tiled(b):
    """Row-major scale bytes [R][S] as tiles of 128 rows x 4 scales."""
    R, S = b.shape
    p = torch.zeros((R + 127) // 128 * 128, S, dtype=torch.uint8, device=b.device)
    p[:R] = b
    return p.view(-1, 4, 32, S // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untiled(t, R, S):
    p = t.view(-1, S // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, S)
    return p[:R]


def _scale_values(byte, fmt):
    if fmt == "mx":
        k = byte.to(torch.int32) - 127
        return _times_pow2(torch.ones_like(k, dtype=torch.float32), k)
    return byte.view(torch.float8_e4m3fn).float()


def _values(code, scale, row, fmt):
    """What the codes stand for, in fp32."""
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                       dtype=torch.float32, device=code.device)
    R, K = code.shape
    v = lut[code.int()].view(R, K // BLOCK[fmt], BLOCK[fmt]) * scale[:, :, None]
    return (v if row is None else v * row[:, None, None]).view(R, K)


def _of_operand(o, fmt, R, K):
    """The fp32 values of a packed operand {"q", "bs", "s"}."""
    byte = _untiled(o["bs"], R, K // BLOCK[fmt]).contiguous()
    return _values(_unpack(o["q"]), _scale_values(byte, fmt), o["s"], fmt)


def _norm(x, res, w):
    """The bf16 residual stream and the fp32 normalised values."""
    s = (x.float() + res.float()).to(torch.bfloat16)
    f = s.float()
    return s, f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS) * w


# ------------------------------------------------------------------ what a program has in hand
def _activations(R, K, g):
    """Hidden states: rows of different size, some channels far larger than the others."""
    x = torch.randn(R, K, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(R, 1, generator=g, device=DEV))
    wide = torch.rand(K, generator=g, device=DEV) < 0.01
    x *= torch.where(wide, 12.0, 1.0)
    return x.to(torch.bfloat16)


def _operand(x, fmt):
    code, scale, row = _quantize(x.float(), fmt)
    return {"q": _pack(code), "bs": _tiled(_scale_bytes(scale, fmt)), "s": row}


def _weights(N, K, fmt, g):
    return _operand(torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K), fmt)


def _room(R, K, fmt):
    """Buffers for a 4-bit matrix."""
    return {"q": torch.empty(R, K // 2, dtype=torch.uint8, device=DEV),
            "bs": torch.empty((R + 127) // 128 * 128 * (K // BLOCK[fmt]), dtype=torch.uint8, device=DEV),
            "s": torch.empty(R, dtype=torch.float32, device=DEV) if fmt == "nv" else None}


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    bf16 = lambda *n: torch.empty(*n, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    st = {"case": c}
    if c["op"] == "quant":
        st["x"] = _activations(c["R"], c["K"], g)
        st["room"] = _room(c["R"], c["K"], c["fmt"])
        st["y"] = bf16(c["R"], c["K"])
        return st
    if c["op"] == "product":
        st["A"] = _operand(_activations(c["M"], c["K"], g), c["fmt"])
        st["B"] = _weights(c["N"], c["K"], c["fmt"], g)
        st["C"] = bf16(c["M"], c["N"])
        return st
    L, d = (c["L"], c["d"]) if c["op"] == "norm" else (c["M"], c["K"])
    st["x"], st["res"] = _activations(L, d, g), _activations(L, d, g)
    st["w"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
    st["sum"] = bf16(L, d)
    if c["op"] == "norm":
        st["q"] = torch.empty(L, d, dtype=torch.float8_e4m3fn, device=DEV)
        st["scale"] = torch.empty(L, dtype=torch.float32, device=DEV)
    else:
        st["room"] = _room(L, d, c["fmt"])
        st["B"] = _weights(c["N"], d, c["fmt"], g)
        st["C"] = bf16(L, c["N"])
    return st


# ------------------------------------------------------------------ one pass
def _run_own(st):
    import joint_audio_video_gb300 as h3
    c = st["case"]
    fmt = {"mx": h3.FP4_MX, "nv": h3.FP4_NV}.get(c.get("fmt"))
    if c["op"] == "quant":
        r = st["room"]
        h3.h3_quantize_rows_fp4(st["x"], fmt, c["R"], c["K"], r["q"], r["bs"], r["s"])
        h3.h3_dequantize_rows_fp4(r["q"], r["bs"], r["s"], fmt, c["R"], c["K"], st["y"])
        return st["y"]
    if c["op"] == "norm":
        h3.h3_rms_norm_fp8(st["x"], st["res"], st["w"], c["L"], c["d"], EPS, st["sum"], st["q"], st["scale"])
        return {"sum": st["sum"], "q": st["q"], "scale": st["scale"]}
    A, B = st.get("A") or st["room"], st["B"]
    if c["op"] == "norm_product":
        h3.h3_rms_norm_fp4(st["x"], st["res"], st["w"], c["M"], c["K"], EPS, fmt, st["sum"], A["q"], A["bs"], A["s"])
    h3.h3_gemm_fp4(A["q"], A["bs"], A["s"], B["q"], B["bs"], B["s"], fmt, c["M"], c["N"], c["K"], st["C"])
    return st["C"] if c["op"] == "product" else {"sum": st["sum"], "C": st["C"]}


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    if c["op"] == "quant":
        return _values(*_quantize(st["x"].float(), c["fmt"]), c["fmt"]).to(torch.bfloat16)
    if c["op"] == "norm":
        s, y = _norm(st["x"], st["res"], st["w"])
        amax = y.abs().amax(1)
        inv = torch.where(amax > 0, 448.0 / amax, torch.ones_like(amax))
        q = (y * inv[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        return {"sum": s, "q": q, "scale": torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))}
    M, N, K, fmt = c["M"], c["N"], c["K"], c["fmt"]
    if c["op"] == "product":
        a, s = _of_operand(st["A"], fmt, M, K), None
    else:
        s, y = _norm(st["x"], st["res"], st["w"])
        a = _values(*_quantize(y, fmt), fmt)
    C = (a @ _of_operand(st["B"], fmt, N, K).T).to(torch.bfloat16)
    return C if s is None else {"sum": s, "C": C}


# ------------------------------------------------------------------ the definitions in 64 bits
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest64(a):
    """The E2M1 magnitude nearest to a >= 0 (fp64), ties to the even code, 6 at most."""
    grid = torch.tensor(_GRID, dtype=torch.float64, device=a.device)
    a = a.clamp(max=6.0)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, 7)
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), grid[hi], grid[lo])


def _e4m3_64(v):
    """The E4M3 value nearest to v in [0, 448] (fp64), ties to even."""
    e = torch.floor(torch.log2(v.clamp(min=2.0 ** -40))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(v / step) * step).clamp(max=448.0)


def _quantized64(x, fmt):
    """The values that fp64 x [R][K] is held as."""
    out = torch.empty_like(x)
    R, K = x.shape
    rows = max(1, 8_000_000 // K)
    for r in range(0, R, rows):
        b = x[r:r + rows].view(-1, K // BLOCK[fmt], BLOCK[fmt])
        amax = b.abs().amax(2, keepdim=True)
        if fmt == "mx":
            k = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 6.0))
            # log2 is rounded: the smallest k with 6 * 2^k >= amax
            k = torch.where(6.0 * torch.exp2(k - 1.0) >= amax, k - 1.0, k)
            k = torch.where(6.0 * torch.exp2(k) < amax, k + 1.0, k)
            scale = torch.exp2(k.clamp(-127.0, 127.0))
        else:
            top = amax.amax(1, keepdim=True)
            k = torch.ceil(torch.log2(top.clamp(min=1e-300) / 2688.0))
            k = torch.where(2688.0 * torch.exp2(k - 1.0) >= top, k - 1.0, k)
            k = torch.where(2688.0 * torch.exp2(k) < top, k + 1.0, k)
            row = torch.where(top > 0, torch.exp2(k.clamp(-126.0, 126.0)), torch.ones_like(top))
            scale = _e4m3_64(amax / (6.0 * row)) * row
        live = scale > 0
        v = torch.where(live, b.abs() / torch.where(live, scale, torch.ones_like(scale)), torch.zeros_like(b))
        out[r:r + rows] = (torch.copysign(_nearest64(v), b) * scale).view(-1, K)
    return out


def _operand64(o, fmt, R, K):
    """The fp64 values of a packed operand, read byte by byte from its definition."""
    grid = torch.tensor(_GRID, dtype=torch.float64, device=DEV)
    v = torch.empty(R, K, dtype=torch.float64, device=DEV)
    for half in (0, 1):
        n = (o["q"] >> (4 * half)) & 15
        v[:, half::2] = grid[(n & 7).long()] * torch.where(n >= 8, -1.0, 1.0).double()
    S = K // BLOCK[fmt]
    r = torch.arange(R, device=DEV)[:, None]
    s = torch.arange(S, device=DEV)[None, :]
    at = ((r // 128) * (S // 4) + s // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + s % 4
    byte = o["bs"][at].long()
    if fmt == "mx":
        scale = torch.exp2(byte.double() - 127.0)
    else:
        e, m = byte >> 3 & 15, (byte & 7).double()
        scale = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.exp2(e.double() - 7.0))
    if o["s"] is not None:
        scale = scale * o["s"].double()[:, None]
    return (v.view(R, S, -1) * scale[:, :, None]).view(R, K)


def exact(case, seed):
    c = case
    if "M" in c and 2 * c["M"] * c["N"] * c["K"] > 2e12:
        return None             # minutes in 64 bits
    st = prepare(case, seed)
    if c["op"] == "quant":
        return _quantized64(st["x"].double(), c["fmt"])
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        return _operand64(st["A"], c["fmt"], M, K) @ _operand64(st["B"], c["fmt"], N, K).T
    s = st["x"].double() + st["res"].double()
    # the norm is of the residual stream as it is stored
    f = s.to(torch.bfloat16).double()
    y = f / torch.sqrt((f * f).mean(1, keepdim=True) + EPS) * st["w"].double()
    if c["op"] == "norm":
        scale = y.abs().amax(1) / 448.0
        scale = torch.where(scale > 0, scale, torch.ones_like(scale))
        return {"sum": s, "q": y / scale[:, None], "scale": scale}
    a = _quantized64(y, c["fmt"])
    return {"sum": s, "C": a @ _operand64(st["B"], c["fmt"], c["N"], c["K"]).T}
