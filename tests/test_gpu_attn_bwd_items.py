"""Attention's gradient where a CTA pair takes many items one after another (more than 152 items of
256 tokens of a head, two kinds each), of one to twelve blocks, odd and even numbers of them,
causal (items of different length) and in segments: every head's gradients against a chain in 64
bits with the same roundings, each 128 tokens apart (tests/_rounded.py).  A pair goes from dK and
dV to dQ once, on the way through most of these."""
import pytest
import torch

from tests import _rounded as ro
from tests import _train as tr
from tests.test_gpu_attn_bwd import SCALE, backward, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def heads_forward(qkv, H, seen):
    q, k, v = tr.heads(qkv, H)
    out = [ro.forward_one_head(q[h], k[h], v[h], seen) for h in range(H)]
    return [o for o, _ in out], [s for _, s in out]


@pytest.mark.parametrize("L,H,causal,cu", [
    (700, 40, False, None), (700, 40, True, None), (850, 40, False, None), (897, 33, True, None),
    (1500, 16, False, None), (1500, 40, True, None), (1111, 24, False, [0, 100, 613, 1111]),
    (1290, 40, True, [0, 37, 700, 703, 1290]), (1024, 40, False, [0, 511, 512, 900, 1024]),
    (1025, 31, True, [0, 250, 1025]), (300, 128, False, [0, 7, 300]), (260, 128, True, None)])
def test_items_one_after_another(h3, L, H, causal, cu):
    assert 2 * ((L + 255) // 256) * H > 152
    qkv, dO = inputs(L, H, L + H)
    seen = ro.visible(L, causal, cu, DEV)
    O, lse = heads_forward(qkv, H, seen)
    got = backward(h3, qkv, torch.cat(O, 1).to(torch.bfloat16), torch.stack(lse).float(), dO, H, causal, cu,
                   SCALE).view(L, 3, H, 128)
    at = torch.arange(L, device=DEV)
    for h in range(H):
        ro.check_head(got[:, :, h].transpose(0, 1).double(), at, ro.head_of(qkv, dO, h, H), seen,
                      what=f"L={L} head {h} of {H} causal={causal} cu={cu}", OL=(O[h], lse[h]))
