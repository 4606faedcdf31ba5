"""The rotation's sine and cosine in the norm of queries and keys and in its gradient, for
elements that come from one of them alone: a pair (0, v) turned by a is (-v sin a, v cos a), so a
small sine is not hidden behind the other term.  fp32 functions and arithmetic: each element is
right to one rounding to bf16 and, before it, 2^-16 of itself (the mean of 128 squares 2^-17 at
most, half of it in the root; the root, the sine, the angle, three products: 2^-21 together)."""
import pytest
import torch

from tests import _train as tr
from tests.test_gpu_qk_norm import norm, norm_bwd

pytestmark = pytest.mark.gpu
DEV = "cuda"


def within(got, ref, what):
    tr.assert_within(got, ref, (tr.U + (1 + tr.U) * 2.0 ** -16) * ref.abs() + 2.0 ** -133, what)


@pytest.mark.parametrize("base,sec", [(1e4, (32, 48, 48)), (1e6, (32, 48, 48)), (1e4, (128, 0, 0)),
                                      (5e8, (42, 44, 42))])
@pytest.mark.parametrize("H", [1, 3])
def test_a_small_sine_keeps_its_bits(h3, H, base, sec):
    L, eps = 97, 1e-6
    g = torch.Generator().manual_seed(H)
    odd = torch.arange(128) % 2 == 1
    qkv = torch.randn(L, 3 * H, 128, generator=g).clamp(min=-2, max=2) * odd
    dout = torch.randn(L, 3 * H, 128, generator=g) * odd
    qkv, dout = (t.view(L, -1).to(torch.bfloat16).to(DEV) for t in (qkv, dout))
    wq, wk = ((1 + 0.3 * torch.randn(128, generator=g)).to(DEV) for _ in range(2))
    pos = torch.randint(-3, 60, (L, 3), generator=g, dtype=torch.int32)
    pos[:4] = torch.tensor([[1, 1, 1], [-1, -1, -1], [2, 2, 2], [0, 0, 0]])
    pos = pos.to(DEV)
    ref, _ = tr.qk_norm(qkv, pos, wq, wk, H, eps, sec, base)
    within(norm(h3, qkv, pos, wq, wk, H, eps, sec=sec, base=base), ref, "norm")
    # x r^2 mean(x g w) is zero where x is: the even elements of the gradient are r w v sin a
    (dx, _, _), _ = tr.qk_norm_bwd(qkv, pos, wq, wk, dout, H, eps, sec, base)
    got, _, _ = norm_bwd(h3, qkv, pos, wq, wk, dout, H, eps, sec=sec, base=base)
    within(got[:, 0::2], dx[:, 0::2], "gradient")
