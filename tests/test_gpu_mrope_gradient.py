"""The gradient of the rotation alone: h3_mrope_apply with negated positions, since a turn's
transpose is the turn back.  Bound: one rounding to bf16, and before it an angle rounded to fp32
twice and fp32 functions (2^-23 of the angle and 2^-21) on the pair's magnitude."""
import pytest
import torch

from tests import _train as tr
from tests.test_gpu_qk_norm import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L,H", [(1, 1), (77, 3), (1030, 5)])
def test_negated_positions_turn_back(h3, L, H):
    _, pos, _, _, dout = inputs(L, H, L)
    got = dout.clone()
    h3.h3_mrope_apply(got, -pos, L, H)
    assert h3.h3_sync_status() == 0
    x = dout.double().view(L, 3, H, 128)
    ang = tr.angles(pos, (32, 48, 48), 1e4)
    ref = tr.turn(x[:, :2], -ang)
    pair = x[:, :2].reshape(L, 2, H, 64, 2).abs().sum(4, keepdim=True).expand(-1, -1, -1, -1, 2).reshape(ref.shape)
    off = (2.0 ** -23 * ang.abs() + 2.0 ** -21)[:, None, None].repeat_interleave(2, 3)
    bound = tr.U * ref.abs() + (1 + tr.U) * off * pair + 2.0 ** -133
    tr.assert_within(got.view(L, 3, H, 128)[:, :2], ref, bound, f"L={L} H={H}")
    assert torch.equal(got.view(L, 3, H, 128)[:, 2], dout.view(L, 3, H, 128)[:, 2])
