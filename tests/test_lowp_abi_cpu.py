"""The 4-bit projections and the quantising norms on a machine without a GPU: the library
exports what include/h3attn_lowp.h declares and refuses bad arguments before any launch."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, WS = 1, 6
P = 1 << 30          # an aligned fake address: never dereferenced on these paths
FAR = 1 << 36        # arrays this far apart do not overlap


@pytest.fixture(scope="module")
def lib():
    from joint_audio_video_gb300 import build
    build.build()
    import joint_audio_video_gb300 as h3
    return h3


def at(i):
    return P + i * FAR


def test_library_exports_every_declared_entry_point(lib):
    with open(os.path.join(ROOT, "include", "h3attn_lowp.h")) as f:
        names = sorted(set(re.findall(r"^\s*h3_status\s+(h3_\w+)\s*\(", f.read(), re.M)))
    assert sorted(lib.LOWP_SYMBOLS) == names and len(names) == 8
    raw = ctypes.CDLL(lib.lib_path)
    for n in names:
        assert hasattr(raw, n) and n in lib.__all__


def test_scale_bytes(lib):
    assert lib.h3_fp4_scale_bytes(lib.FP4_MX, 1, 128) == 128 * 4
    assert lib.h3_fp4_scale_bytes(lib.FP4_NV, 129, 128) == 256 * 8
    assert lib.h3_fp4_scale_bytes(lib.FP4_NV, 58758, 5120) == 58880 * 320
    # more than 2^32 bytes
    assert lib.h3_fp4_scale_bytes(lib.FP4_NV, 2 ** 31 - 1, 65536) == 2 ** 31 * 4096
    L = lib.load()
    n = ctypes.c_size_t(0)
    for fmt, R, K in ((0, 8, 128), (3, 8, 128), (1, 0, 128), (1, -1, 128), (1, 8, 64), (1, 8, 0),
                      (1, 8, 200), (1, 8, 65536 + 128), (1, 8, -128)):
        assert L.h3_fp4_scale_bytes(fmt, R, K, ctypes.byref(n)) == INV
    assert L.h3_fp4_scale_bytes(1, 8, 128, None) == INV


@pytest.mark.parametrize("fmt", [1, 2])
def test_quantiser_refusals(lib, fmt):
    L = lib.load()

    def call(x=at(0), f=fmt, R=64, K=256, q=at(1), bs=at(2), s=at(3)):
        return L.h3_quantize_rows_fp4(x, f, R, K, q, bs, s, None)
    for bad in (dict(f=0), dict(f=3), dict(R=0), dict(R=-5), dict(K=0), dict(K=192), dict(K=65664),
                dict(x=None), dict(q=None), dict(bs=None), dict(x=at(0) + 8), dict(q=at(1) + 4),
                dict(bs=at(2) + 1), dict(q=at(0)), dict(q=at(0) + 64 * 512 - 16),
                dict(bs=at(0) + 16), dict(bs=at(1) + 16)):
        assert call(**bad) == INV, bad
    if fmt == 2:       # row factors are written
        for bad in (dict(s=None), dict(s=at(3) + 2), dict(s=at(0) + 64), dict(s=at(2))):
            assert call(**bad) == INV, bad

    def back(q=at(1), bs=at(2), s=at(3), f=fmt, R=64, K=256, y=at(0)):
        return L.h3_dequantize_rows_fp4(q, bs, s, f, R, K, y, None)
    for bad in (dict(f=0), dict(R=0), dict(K=100), dict(q=None), dict(bs=None), dict(y=None),
                dict(s=at(3) + 1), dict(y=at(1)), dict(y=at(2) + 16), dict(y=at(3)),
                dict(q=at(1) + 8), dict(y=at(0) + 2)):
        assert back(**bad) == INV, bad


def test_product_refusals(lib):
    L = lib.load()

    def call(A=at(0), abs_=at(1), as_=at(2), B=at(3), bbs=at(4), bs_=at(5), fmt=1, M=64, N=256,
             K=256, C=at(6)):
        return L.h3_gemm_fp4(A, abs_, as_, B, bbs, bs_, fmt, M, N, K, C, None)
    for bad in (dict(fmt=0), dict(fmt=4), dict(M=0), dict(N=0), dict(N=192), dict(K=64),
                dict(K=320), dict(K=65664), dict(A=None), dict(abs_=None), dict(B=None),
                dict(bbs=None), dict(C=None), dict(A=at(0) + 8), dict(abs_=at(1) + 8),
                dict(as_=at(2) + 4), dict(B=at(3) + 2), dict(bbs=at(4) + 4), dict(bs_=at(5) + 8),
                dict(C=at(6) + 2), dict(C=at(0)), dict(C=at(1)), dict(C=at(2)), dict(C=at(3)),
                dict(C=at(4)), dict(C=at(5)), dict(M=2 ** 31 - 1, N=2 ** 31 - 128, K=128)):
        assert call(**bad) == INV, bad


def test_norm_refusals(lib):
    L = lib.load()

    def n8(x=at(0), res=at(1), w=at(2), n=64, d=256, eps=1e-6, sum=at(3), q=at(4), scale=at(5)):
        return L.h3_rms_norm_fp8(x, res, w, n, d, eps, sum, q, scale, None)

    def n4(x=at(0), res=at(1), w=at(2), n=64, d=256, eps=1e-6, sum=at(3), q=at(4), fmt=2,
           bs=at(6), scale=at(5)):
        return L.h3_rms_norm_fp4(x, res, w, n, d, eps, fmt, sum, q, bs, scale, None)
    for call in (n8, n4):
        for bad in (dict(n=0), dict(d=0), dict(d=200), dict(d=16512), dict(eps=-1.0),
                    dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(w=None),
                    dict(q=None), dict(scale=None), dict(x=at(0) + 2), dict(res=at(1) + 8),
                    dict(w=at(2) + 4), dict(sum=at(3) + 4), dict(q=at(4) + 8),
                    dict(scale=at(5) + 1), dict(q=at(0)), dict(q=at(1)), dict(q=at(2)),
                    dict(q=at(3)), dict(scale=at(0)), dict(scale=at(3)), dict(scale=at(4)),
                    dict(sum=at(0) + 16), dict(sum=at(1) + 512), dict(sum=at(2))):
            assert call(**bad) == INV, (call.__name__, bad)
    for bad in (dict(fmt=0), dict(fmt=3), dict(bs=None), dict(bs=at(6) + 8), dict(bs=at(0)),
                dict(bs=at(4)), dict(bs=at(3))):
        assert n4(**bad) == INV, bad


def test_mlp_refusals_and_workspace(lib):
    L = lib.load()
    r = lambda n: (n + 255) // 256 * 256  # noqa: E731
    desc = lib.MlpDesc.make(L=300, d=256, hidden=1024)
    for fmt, blk in ((1, 32), (2, 16)):
        assert lib.h3_mlp_workspace_size_fp4(desc, fmt) == (
            lib.h3_mlp_workspace_size(desc) + r(300 * 512) + r(384 * 1024 // blk) + r(300 * 4))
    n = ctypes.c_size_t(0)
    assert L.h3_mlp_workspace_size_fp4(ctypes.byref(desc), 0, ctypes.byref(n)) == INV
    assert L.h3_mlp_workspace_size_fp4(ctypes.byref(desc), 1, None) == INV
    for bad in (dict(L=0), dict(d=200), dict(hidden=100), dict(hidden=65664), dict(n_mod=0),
                dict(ln_eps=-1.0)):
        b = lib.MlpDesc.make(**{**dict(L=300, d=256, hidden=1024), **bad})
        assert L.h3_mlp_workspace_size_fp4(ctypes.byref(b), 1, ctypes.byref(n)) == INV
    need = lib.h3_mlp_workspace_size_fp4(desc, 2)
    names = ("x", "mod", "shift", "scale", "gate", "W1_q", "W1_bs", "W1_s", "W2_q", "W2_bs", "W2_s")

    def call(fmt=2, nbytes=need, ws=at(20), out=at(21), **kw):
        a = {k: at(i) for i, k in enumerate(names)} | kw
        return L.h3_mlp_block_fwd_fp4(ctypes.byref(desc), fmt, *[a[k] for k in names], ws, nbytes,
                                      out, None)
    assert call(nbytes=need - 1) == WS
    for k in names:
        if not k.endswith("_s"):
            assert call(**{k: None}) == INV
        if k != "mod":
            assert call(**{k: at(3) + 8}) == INV
        assert call(ws=at(names.index(k))) == INV
    for bad in (dict(fmt=0), dict(ws=None), dict(ws=at(20) + 16), dict(out=None), dict(out=at(20)),
                dict(out=at(0) + 16), dict(out=at(5)), dict(out=at(2))):
        assert call(**bad) == INV, bad
