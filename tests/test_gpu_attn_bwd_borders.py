"""Attention's gradient with segments that begin and end at every remainder of four tokens (lse and D
come in groups of four, blocks of 128), where an item's first or last block is moved inside its
segments: against the definitions in 64 bits, and through the checked build."""
import pytest
import torch

import joint_audio_video_gb300 as h3lib
from tests.test_gpu_attn_bwd import SCALE, check_case, forward, inputs
from tests.test_gpu_checked import _both, checked  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("a", [256, 257, 258, 259, 383, 386, 509, 511])
@pytest.mark.parametrize("b", [897, 898, 899, 900, 1023, 1025])
def test_borders(h3, a, b, causal):
    check_case(h3, 1300, 1, causal, [0, a, b, 1300], seed=a + b)


@pytest.mark.parametrize("cu", [[0, 2, 1201, 1203], [0, 1, 600, 1199, 1200], [0, 3, 3, 258, 261, 517, 902],
                                [0, 130, 387, 644, 901], [0, 767, 769, 1030]])
def test_short_segments_beside_long_ones(h3, cu):
    for causal in (False, True):
        check_case(h3, cu[-1], 2, causal, cu, seed=cu[-1])


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("cu", [[0, 770, 1101, 1600], [0, 3, 515, 1030, 1031], [0, 259, 600, 1501]])
def test_checked_build_reports_nothing(h3, checked, cu, causal):  # noqa: F811
    L, H = cu[-1], 2
    qkv, dO = inputs(L, H, L)
    O, lse = forward(qkv, H, bool(causal), cu)

    def run():
        n = h3lib.h3_attn_bwd_workspace_size(L, H)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        out = torch.zeros_like(qkv)
        h3lib.h3_joint_attn_varlen_bwd(qkv, O, lse, dO, cu, L, H, 128, causal, SCALE, ws, n, out)
        return (out,)

    _both(checked, run)
