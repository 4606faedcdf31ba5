"""Attention's gradient over all tokens of a full-size request, one head: sampled tokens against a
chain in 64 bits with the same roundings, in the 2-norm, where one block of 128 tokens left out
of the 460 would show (tests/_rounded.py; tests/test_rounded_chain_cpu.py plants it)."""
import pytest
import torch

from tests import _rounded as ro
from tests.test_gpu_attn_bwd import backward, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("causal,cu", [(False, None), (True, None), (False, [0, 358, 57958, 58758])])
def test_sampled_tokens_of_a_full_size_request(h3, causal, cu):
    L = 58758
    qkv, dO = inputs(L, 1, 18, d_scale=0.1)
    head = ro.head_of(qkv, dO, 0, 1)
    seen = ro.visible(L, causal, cu, DEV)
    O, lse = ro.forward_one_head(*head[:3], seen)
    got = backward(h3, qkv, O.to(torch.bfloat16), lse.float()[None].contiguous(), dO, 1, causal, cu)
    # a group of 16 tokens from each of the places where items and blocks begin and end; each
    # group's gradients are compared apart
    starts = torch.tensor([0, 120, 250, 350, 504, 9000, 29111, 45055, 57950, 58616, L - 16])
    at = (starts[:, None] + torch.arange(16)).flatten().to(DEV)
    mine = got.view(L, 3, 128)[at].transpose(0, 1).double()
    ro.check_head(mine, at, head, seen, what=f"causal={causal} cu={cu}", rows=16, OL=(O, lse))
