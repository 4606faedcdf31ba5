"""Attention's causal gradient on both sides of the limit between the orders of its items (192 MB
of streams at 1 KB a token and head: by rows of all heads below it, head by head beyond): an
item's result does not depend on the order, so a head has the bits of a call of its own, and the
64-bit chain's gradients (tests/_rounded.py)."""
import pytest
import torch

from tests import _rounded as ro
from tests.test_gpu_attn_bwd import SCALE, backward, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("L,H,cu", [(4099, 47, None), (4099, 48, None), (12300, 17, None),
                                    (4099, 50, [0, 1000, 1001, 3333, 4099])])
def test_a_head_does_not_depend_on_the_order(h3, L, H, cu):
    qkv, dO = inputs(L, H, H)
    O = torch.empty(L, H * 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(H, L, device=DEV)
    if cu is None:
        h3.h3_joint_attn_fwd(qkv, L, H, 128, True, SCALE, O, lse)
    else:
        h3.h3_joint_attn_varlen_fwd(qkv, cu, L, H, 128, True, SCALE, O, lse)
    seen = ro.visible(L, True, cu, DEV)
    picked = (0, 1, H // 2, H - 1)
    for h in (0, H - 1):   # O and lse of the compared heads from 64 bits
        o, s = ro.forward_one_head(*ro.head_of(qkv, dO, h, H)[:3], seen)
        O[:, 128 * h:128 * h + 128], lse[h] = o.to(torch.bfloat16), s.float()
    got = backward(h3, qkv, O, lse, dO, H, True, cu).view(L, 3, H, 128)
    for h in picked:
        one = qkv.view(L, 3, H, 128)[:, :, h].reshape(L, 384)
        cols = slice(128 * h, 128 * h + 128)
        alone = backward(h3, one, O[:, cols].contiguous(), lse[h:h + 1].contiguous(), dO[:, cols].contiguous(),
                         1, True, cu)
        assert torch.equal(got[:, :, h].reshape(L, 384), alone), f"head {h}"
    at = torch.arange(L, device=DEV) if L < 5000 else torch.arange(0, L, 7, device=DEV)
    for h in (0, H - 1):
        ro.check_head(got[:, :, h].transpose(0, 1)[:, at].double(), at, ro.head_of(qkv, dO, h, H), seen,
                      what=f"L={L} head {h} of {H} cu={cu}")
