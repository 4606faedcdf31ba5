"""Attention's gradient against the definitions in 64 bits (element-wise bounds from counted
roundings, tests/_train.py), at lengths around every tile border, causal and with segments;
determinism, streams, graphs, canaries, offsets past 32 bits."""
import math

import pytest
import torch

import joint_audio_video_gb300 as h3lib
from tests import _train as tr
from tests.test_gpu_checked import _both, checked  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1 / math.sqrt(128)


def inputs(L, H, seed, q_scale=1.0, d_scale=1.0):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(L, 3 * H * 128, generator=g)
    qkv[:, :H * 128] *= q_scale
    dO = d_scale * torch.randn(L, H * 128, generator=g)
    return qkv.to(torch.bfloat16).to(DEV), dO.to(torch.bfloat16).to(DEV)


def forward(qkv, H, causal=False, cu=None, scale=SCALE):
    """What the forward pass leaves, rounded from 64 bits."""
    O, lse = tr.attention(qkv, H, causal, cu, scale)
    return O.to(torch.bfloat16), lse.float().contiguous()


def backward(h3, qkv, O, lse, dO, H, causal=False, cu=None, scale=SCALE, check=True):
    L = qkv.shape[0]
    n = h3.h3_attn_bwd_workspace_size(L, H)
    pad = 4096
    room = torch.full((n + 2 * pad,), 0x5A, dtype=torch.uint8, device=DEV)
    ws = room[pad:pad + n]
    band = torch.full((L + 2, 3 * H * 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    out = band[1:L + 1]
    if cu is None:
        h3.h3_joint_attn_bwd(qkv, O, lse, dO, L, H, 128, causal, scale, ws, n, out)
    else:
        h3.h3_joint_attn_varlen_bwd(qkv, O, lse, dO, cu, L, H, 128, causal, scale, ws, n, out)
    if check:
        assert h3.h3_sync_status() == 0
        assert torch.isnan(band[0]).all() and torch.isnan(band[-1]).all()
        assert (room[:pad] == 0x5A).all() and (room[pad + n:] == 0x5A).all()
    return out


def check_case(h3, L, H, causal, cu=None, seed=0, scale=SCALE, **kw):
    qkv, dO = inputs(L, H, seed, **kw)
    O, lse = forward(qkv, H, causal, cu, scale)
    got = backward(h3, qkv, O, lse, dO, H, causal, cu, scale)
    ref, bound = tr.attention_bwd(qkv, dO, H, causal, cu, scale)
    return tr.assert_within(got, ref, bound, f"L={L} H={H} causal={causal} cu={cu}")


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("L", [1, 2, 5, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 385, 512,
                               641, 1000, 1537])
def test_lengths(h3, L, causal):
    check_case(h3, L, 1 + L % 3, causal, seed=L)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("cu", [[0, 10, 30], [0, 7, 7, 130, 300, 301, 700], [0, 0, 1, 1],
                                [0, 511, 513, 1025, 1537], [0, 256, 512, 1000],
                                [0, 1, 2, 3, 4, 5, 6, 130], list(range(0, 65 * 9, 9)),
                                [0, 129, 1151, 1151]])
def test_segments(h3, cu, causal):
    check_case(h3, cu[-1], 2, causal, cu, seed=len(cu))


@pytest.mark.parametrize("H", [1, 5, 16, 40, 128])
def test_head_counts(h3, H):
    check_case(h3, 200, H, False, seed=H)
    check_case(h3, 140, H, True, cu=[0, 33, 140], seed=H)


@pytest.mark.parametrize("kw", [dict(q_scale=8.0), dict(q_scale=40.0), dict(q_scale=0.0),
                                dict(d_scale=2.0 ** 40), dict(d_scale=2.0 ** -60),
                                dict(d_scale=0.0), dict(scale=1.0), dict(scale=2.0 ** -12)])
def test_sharp_flat_and_far_values(h3, kw):
    for causal in (False, True):
        check_case(h3, 300, 2, causal, seed=7, **kw)


def test_a_bad_value_stays_in_its_head(h3):
    """A NaN in one head's value, an infinity in another's gradient: the third head's bits stay."""
    L, H = 300, 3
    qkv, dO = inputs(L, H, 13)
    O, lse = forward(qkv, H)
    ref = backward(h3, qkv, O, lse, dO, H).clone()
    bad, g = qkv.clone(), dO.clone()
    bad[7, 2 * H * 128 + 3] = float("nan")
    g[200, 128 + 5] = float("inf")
    got = backward(h3, bad, O, lse, g, H)
    third = (torch.arange(3 * H * 128, device=DEV) // 128) % H == 2
    assert torch.equal(got[:, third], ref[:, third])
    assert torch.isnan(got[:, :128]).any() and not torch.isfinite(got[:, 128:256]).all()


def test_zero_gradient_gives_zeros(h3):
    qkv, dO = inputs(333, 2, 1)
    O, lse = forward(qkv, 2)
    assert (backward(h3, qkv, O, lse, torch.zeros_like(dO), 2) == 0).all()


def test_what_the_forward_call_leaves_is_taken(h3):
    L, H = 1111, 3
    for causal, cu in ((False, None), (True, None), (False, [0, 100, 613, L])):
        qkv, dO = inputs(L, H, 9)
        O = torch.empty(L, H * 128, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(H, L, device=DEV)
        if cu is None:
            h3.h3_joint_attn_fwd(qkv, L, H, 128, causal, SCALE, O, lse)
        else:
            h3.h3_joint_attn_varlen_fwd(qkv, cu, L, H, 128, causal, SCALE, O, lse)
        got = backward(h3, qkv, O, lse, dO, H, causal, cu)
        # the forward pass rounds P to bf16 on its way into P V
        q, k, v = tr.heads(qkv, H)
        p = torch.exp((q @ k.transpose(1, 2)) * SCALE - tr.attention(qkv, H, causal, cu)[1][:, :, None])
        p = p.masked_fill(tr.hidden(L, cu, causal, DEV), 0.0)
        off = ((tr.U + 2.0 ** -12) * p @ v.abs()).transpose(0, 1).reshape(L, -1)
        ref, bound = tr.attention_bwd(qkv, dO, H, causal, cu, dO_of=off)
        tr.assert_within(got, ref, bound, f"after the forward call, causal={causal} cu={cu}")


def test_one_segment_equals_the_whole_bitwise(h3):
    qkv, dO = inputs(777, 2, 3)
    for causal in (False, True):
        O, lse = forward(qkv, 2, causal)
        a = backward(h3, qkv, O, lse, dO, 2, causal)
        b = backward(h3, qkv, O, lse, dO, 2, causal, [0, 777])
        assert torch.equal(a, b)


def test_segments_equal_their_own_calls(h3):
    """Rows of one segment see nothing of the others: values (NaN apart) elsewhere do not matter."""
    H, cu = 2, [0, 256, 1024]
    qkv, dO = inputs(1024, H, 4)
    O, lse = forward(qkv, H, cu=cu)
    whole = backward(h3, qkv, O, lse, dO, H, cu=cu)
    for a, b in zip(cu, cu[1:]):
        part = backward(h3, qkv[a:b].clone(), O[a:b].clone(), lse[:, a:b].contiguous(), dO[a:b].clone(), H)
        assert torch.equal(whole[a:b], part)


def test_arrays_on_sixteen_byte_boundaries(h3):
    """Every array 16 bytes past a larger boundary: the bits of aligned ones."""
    L, H = 400, 2
    qkv, dO = inputs(L, H, 12)
    O, lse = forward(qkv, H)
    ref = backward(h3, qkv, O, lse, dO, H).clone()

    def moved(t):
        room = torch.empty(t.numel() + 16 // t.element_size(), dtype=t.dtype, device=DEV)
        m = room[16 // t.element_size():].view(t.shape)
        m.copy_(t)
        assert m.data_ptr() % 32 == 16
        return m

    out = moved(torch.full_like(qkv, float("nan")))
    n = h3.h3_attn_bwd_workspace_size(L, H)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    h3.h3_joint_attn_bwd(moved(qkv), moved(O), moved(lse), moved(dO), L, H, 128, False, SCALE, ws, n, out)
    assert h3.h3_sync_status() == 0
    assert torch.equal(out, ref)


def test_same_bits_every_time_on_any_stream(h3):
    L, H = 1300, 4
    qkv, dO = inputs(L, H, 5)
    O, lse = forward(qkv, H, True)
    ref = backward(h3, qkv, O, lse, dO, H, True).clone()
    n = h3.h3_attn_bwd_workspace_size(L, H)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.full_like(ref, float("nan")) for _ in streams]
    rooms = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o, w in zip(streams, outs, rooms):   # overlapping calls, a workspace each
            h3.h3_joint_attn_bwd(qkv, O, lse, dO, L, H, 128, True, SCALE, w, n, o, stream=s)
    torch.cuda.synchronize()
    assert h3.h3_sync_status() == 0
    assert all(torch.equal(o, ref) for o in outs)


def test_captured_and_replayed(h3):
    L, H = 500, 2
    qkv, dO = inputs(L, H, 6)
    O, lse = forward(qkv, H)
    ref = backward(h3, qkv, O, lse, dO, H).clone()
    n = h3.h3_attn_bwd_workspace_size(L, H)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        h3.h3_joint_attn_bwd(qkv, O, lse, dO, L, H, 128, False, SCALE, ws, n, out)
    for _ in range(3):
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    # new inputs in the same arrays
    qkv2, dO2 = inputs(L, H, 16)
    O2, lse2 = forward(qkv2, H)
    for a, b in ((qkv, qkv2), (dO, dO2), (O, O2), (lse, lse2)):
        a.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    assert h3.h3_sync_status() == 0
    r, bound = tr.attention_bwd(qkv2, dO2, H)
    tr.assert_within(out, r, bound, "replayed on other inputs")


def test_offsets_past_32_bits(h3):
    """More than 2^32 elements of qkv: the last segment's rows against the definitions."""
    L, H = 290_000, 40
    cu = [L * i // 60 for i in range(60)] + [L - 150, L]
    a = cu[-2]
    g = torch.Generator(device=DEV).manual_seed(1)
    qkv = torch.zeros(L, 3 * H * 128, dtype=torch.bfloat16, device=DEV)
    O, dO = (torch.zeros(L, H * 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    lse = torch.zeros(H, L, device=DEV)
    assert qkv.numel() > 2 ** 32
    qkv[a:].copy_(torch.randn(150, 3 * H * 128, generator=g, device=DEV))
    dO[a:].copy_(torch.randn(150, H * 128, generator=g, device=DEV))
    o, l = forward(qkv[a:], H)
    O[a:], lse[:, a:] = o, l
    n = h3.h3_attn_bwd_workspace_size(L, H)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out = torch.full_like(qkv, float("nan"))
    h3.h3_joint_attn_varlen_bwd(qkv, O, lse, dO, cu, L, H, 128, False, SCALE, ws, n, out)
    assert h3.h3_sync_status() == 0
    ref, bound = tr.attention_bwd(qkv[a:], dO[a:], H)
    tr.assert_within(out[a:], ref, bound, "last segment")
    assert (out[:a] == 0).all()


def test_full_length_rows(h3):
    """All tokens of a full-size request, one head: sampled rows and keys in 64 bits."""
    L = 58758
    qkv, dO = inputs(L, 1, 8, d_scale=0.1)
    q, k, v = (t[0] for t in tr.heads(qkv, 1))
    g = tr.heads(dO, 1)[0][0]
    O, lse = [], []
    for i in range(0, L, 2048):
        s = (q[i:i + 2048] @ k.T) * SCALE
        lse.append(torch.logsumexp(s, 1))
        O.append(torch.exp(s - lse[-1][:, None]) @ v)
    O, lse = torch.cat(O), torch.cat(lse)
    got = backward(h3, qkv, O.to(torch.bfloat16), lse.float()[None].contiguous(), dO, 1).double()
    at = torch.tensor([0, 1, 127, 128, 255, 256, 29000, 58623, 58624, L - 2, L - 1], device=DEV)
    D = (g * O).sum(1)
    off_D = tr.U * (g.abs() * O.abs()).sum(1)
    # dQ: rows of S
    p = torch.exp((q[at] @ k.T) * SCALE - lse[at, None])
    ds = p * (g[at] @ v.T - D[at, None])
    off = tr.U * ds.abs() + p * (off_D[at, None] + tr.F * (g[at].abs() @ v.abs().T))
    tr.assert_within(got[at, :128], SCALE * ds @ k,
                     1.1 * SCALE * off @ k.abs() + tr.U * (SCALE * ds @ k).abs(), "dQ rows")
    # dK, dV: columns of S
    p = torch.exp((k[at] @ q.T) * SCALE - lse[None])
    ds = p * (v[at] @ g.T - D[None])
    off = tr.U * ds.abs() + p * (off_D[None] + tr.F * (v[at].abs() @ g.abs().T))
    tr.assert_within(got[at, 128:256], SCALE * ds @ q,
                     1.1 * SCALE * off @ q.abs() + tr.U * (SCALE * ds @ q).abs(), "dK rows")
    tr.assert_within(got[at, 256:], p @ g, 1.1 * tr.U * p @ g.abs() + tr.U * (p @ g).abs(), "dV rows")


@pytest.mark.parametrize("L,H,causal,cu", [(1, 1, 0, None), (130, 2, 1, None), (700, 3, 0, None),
                                           (391, 2, 1, [0, 5, 5, 200, 391])])
def test_checked_build_reports_nothing(h3, checked, L, H, causal, cu):  # noqa: F811
    qkv, dO = inputs(L, H, L)
    O, lse = forward(qkv, H, bool(causal), cu)

    def run():
        n = h3lib.h3_attn_bwd_workspace_size(L, H)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        out = torch.zeros_like(qkv)
        if cu is None:
            h3lib.h3_joint_attn_bwd(qkv, O, lse, dO, L, H, 128, causal, SCALE, ws, n, out)
        else:
            h3lib.h3_joint_attn_varlen_bwd(qkv, O, lse, dO, cu, L, H, 128, causal, SCALE, ws, n, out)
        return (out,)

    _both(checked, run)
