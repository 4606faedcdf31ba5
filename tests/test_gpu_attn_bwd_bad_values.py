"""How far a bad value reaches in attention's gradient with segments: in its own head, the blocks
of 256 tokens that hold a token of its segment, and nothing else, wherever segments begin and
end.  Every other gradient keeps its bits."""
import pytest
import torch

from tests.test_gpu_attn_bwd import backward, forward, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def reach(cu, t):
    """Truth for each token: in a block of 256 that holds a token of t's segment."""
    a, b = next((a, b) for a, b in zip(cu, cu[1:]) if a <= t < b)
    n = torch.arange(cu[-1], device=DEV) // 256
    return (n >= a // 256) & (n <= (b - 1) // 256)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("cu,t", [
    # just past the end of a segment whose first token is on no 128-row boundary
    ([0, 100, 512, 1024], 512), ([0, 100, 512, 1024], 600), ([0, 100, 512, 1024], 639),
    ([0, 3, 768, 1300], 768), ([0, 3, 768, 1300], 770), ([0, 255, 511, 1024, 1100], 1024),
    # a segment that ends inside a block of 256, one segment on
    ([0, 100, 300, 520, 1024], 600), ([0, 1, 2, 515, 1290], 516),
    # one to three tokens ahead of a segment's first
    ([0, 770, 1100, 1600], 769), ([0, 770, 1100, 1600], 768), ([0, 259, 600, 1501], 258),
    ([0, 257, 1501], 256), ([0, 511, 1030, 1501], 510),
    # the last segment, the first one, an empty one beside it
    ([0, 256, 256, 900, 901], 900), ([0, 130, 130, 700], 129)])
def test_a_bad_value_stays_near_its_segment(h3, cu, t, causal):
    L, H = cu[-1], 2
    qkv, dO = inputs(L, H, t)
    O, lse = forward(qkv, H, causal, cu)
    ref = backward(h3, qkv, O, lse, dO, H, causal, cu).clone()
    assert torch.isfinite(ref).all()
    keep = torch.ones(L, 3, H, 128, dtype=torch.bool, device=DEV)
    keep[:, :, 1] = ~reach(cu, t)[:, None, None]
    keep = keep.view(L, -1)
    assert not keep.all() and (keep[:, 128:256].any() or L // 256 < 3)
    d = H * 128
    for what, at, value in (("Q", 128, NAN), ("K", d + 128 + 7, INF), ("V", 2 * d + 128 + 99, NAN),
                            ("O", 128 + 5, NAN), ("dO", 128 + 64, -INF), ("lse", 0, NAN), ("lse", 0, -INF)):
        x = [a.clone() for a in (qkv, O, lse, dO)]
        if what == "lse":
            x[2][1, t] = value
        else:
            x[{"O": 1, "dO": 3}.get(what, 0)][t, at] = value
        got = backward(h3, x[0], x[1], x[2], x[3], H, causal, cu)
        lost = ~(got.view(torch.int16) == ref.view(torch.int16)) & keep
        rows = lost.any(1).nonzero().flatten().tolist()
        assert not rows, f"{what} of token {t}, cu={cu}: tokens {rows[0]} .. {rows[-1]} ({len(rows)})"
