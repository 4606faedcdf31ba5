"""The comparison of tests/_rounded.py on a machine without a GPU: a chain computed in 32 bits
passes it; blocks of rows left out of the sums, even one of 460, do not, although element-wise
bounds over as many terms take them."""
import pytest
import torch

from tests import _rounded as ro
from tests import _train as tr


def sampled(L, at, seed):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(L, 128, generator=g).to(torch.bfloat16).double() for _ in range(3))
    dO = (0.1 * torch.randn(L, 128, generator=g)).to(torch.bfloat16).double()
    # O and lse of the right size without 58,758^2 products; the sums take them as given
    O = torch.randn(L, 128, generator=g, dtype=torch.float64) * (2.7 / L) ** 0.5
    lse = torch.log(torch.tensor(float(L))) + 0.5 + 0.05 * torch.randn(L, generator=g, dtype=torch.float64)
    return q, k, v, dO, O, lse


@pytest.mark.parametrize("L,lost", [(58758, slice(128 * 200, 128 * 201)), (1500, slice(1408, 1500)),
                                    (1111, slice(128, 192))])
def test_a_lost_block_is_refused(L, lost):
    at = torch.tensor([0, 1, 127, 128, 255, 256, L // 2, L - 135, L - 134, L - 2, L - 1])
    q, k, v, g, O, lse = sampled(L, at, L)
    D, Dr = (g * O).sum(1), (g * ro.rnd(O)).sum(1)
    exact = ro.one_head(at, q, k, v, g, lse, D)
    chain = ro.one_head(at, q, k, v, g, lse, Dr, r=ro.rnd)
    # what a kernel does: the same in fp32
    f = lambda x: x.float()  # noqa: E731
    r32 = lambda x: x.to(torch.bfloat16).float()  # noqa: E731
    same = ro.one_head(at, f(q), f(k), f(v), f(g), f(lse), f(Dr), r=r32)
    assert ro.worst_ratio(same, exact, chain)[0] <= 0.8
    wrong = ro.one_head(at, q, k, v, g, lse, Dr, r=ro.rnd, lost=lost)
    assert ro.worst_ratio(wrong, exact, chain)[0] > 2.0
    if L > 50000:   # the element-wise bound over all terms does not see it
        p = torch.exp((k[at] @ q.T) * ro.SCALE - lse[None])
        bound = 1.1 * tr.U * p @ g.abs() + tr.U * exact[2].abs()
        assert ((wrong[2] - exact[2]).abs() <= bound).all()


@pytest.mark.parametrize("causal,cu", [(False, None), (True, None), (False, [0, 40, 40, 170, 300]),
                                       (True, [0, 129, 300])])
def test_the_chain_is_the_definition(causal, cu):
    """Without roundings one_head gives what tests/_train.py has, which is held against differences
    and automatic differentiation; with them it stays within the element-wise bounds."""
    L, H = 300, 2
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(L, 3 * H * 128, generator=g).to(torch.bfloat16)
    dO = torch.randn(L, H * 128, generator=g).to(torch.bfloat16)
    ref, bound = tr.attention_bwd(qkv, dO, H, causal, cu)
    ref, bound = (t.view(L, 3, H, 128) for t in (ref, bound))
    seen = ro.visible(L, causal, cu, "cpu")
    at = torch.arange(L)
    for h in range(H):
        q, k, v, d = ro.head_of(qkv, dO, h, H)
        O, lse = ro.forward_one_head(q, k, v, seen, rows=77)
        exact = ro.one_head(at, q, k, v, d, lse, (d * O).sum(1), seen)
        chain = ro.one_head(at, q, k, v, d, lse, (d * ro.rnd(O)).sum(1), seen, ro.rnd)
        for i in range(3):
            assert float((exact[i] - ref[:, i, h]).abs().max()) <= 1e-12
            assert ((chain[i] - ref[:, i, h]).abs() <= bound[:, i, h]).all()
