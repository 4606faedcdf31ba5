"""The 4-bit MLP sub-block at every number of tokens that takes a product kernel of its own: one
or two rows, few rows (16, 32, 64 columns of the tensor cores, split along K), pairs of CTAs.
Their GELU and gated-residual epilogues are separate code, so each meets the oracle.

Stages are compared as for the other sub-blocks: y with the oracle's, h and out with the oracle
fed the 4-bit operands that the stage before implies as the GPU stored it, at the bf16 bounds.

Against the exact sub-block: the bf16 bounds' error model with the unit roundoff of E2M1, 2^-2
(one mantissa bit), in place of 2^-8: mean relative error 64 x 5e-3 = 0.32, largest error
64 x 2e-2 = 1.28 RMS."""
import math

import numpy as np
import pytest
import torch

import oracle as orc
from tests import _fp4 as f4
from tests._parity import MAX_REL_RMS, MEAN_REL, assert_parity, to64
from tests.test_gpu_fp4 import _guarded, _intact, _quant

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMTS = [f4.MX, f4.NV]
FP4_MAX, FP4_MEAN = 64 * MAX_REL_RMS, 64 * MEAN_REL


class _Mlp:
    def __init__(self, h3, fmt, L, d, hidden, n_mod=3):
        g = torch.Generator().manual_seed(31 * L + hidden + fmt)
        self.h3, self.fmt, self.L, self.d, self.hidden = h3, fmt, L, d, hidden
        self.x = torch.randn(L, d, generator=g).to(torch.bfloat16)
        self.w1 = (torch.randn(hidden, d, generator=g) / math.sqrt(d)).to(torch.bfloat16)
        self.w2 = (torch.randn(d, hidden, generator=g) / math.sqrt(hidden)).to(torch.bfloat16)
        # modalities far apart, so that a row with another's vectors is seen
        self.sh = 0.3 * torch.randn(n_mod, d, generator=g) + torch.arange(n_mod)[:, None] - 1.0
        self.sc = 0.3 * torch.randn(n_mod, d, generator=g)
        self.gt = (0.5 + 0.5 * torch.rand(n_mod, d, generator=g)) * torch.tensor([1.0, -1.0, 0.5])[:n_mod, None]
        self.mod = torch.randint(0, n_mod, (L,), generator=g).to(torch.uint8)
        self.desc = h3.MlpDesc.make(L=L, d=d, hidden=hidden, n_mod=n_mod)
        self.bytes = h3.h3_mlp_workspace_size_fp4(self.desc, fmt)
        self.q1, self.q2 = _quant(h3, self.w1.to(DEV), fmt), _quant(h3, self.w2.to(DEV), fmt)
        self.guard, self.ws = _guarded(self.bytes)

    def run(self, x=None, mod=None, gate=None, out=None):
        x = self.x.to(DEV) if x is None else x
        gout = None
        if out is None:
            gout, out = _guarded(self.L * self.d * 2)
            out = out.view(torch.bfloat16).view(self.L, self.d)
            out.fill_(float("nan"))
        self.h3.h3_mlp_block_fwd_fp4(
            self.desc, self.fmt, x, (self.mod if mod is None else mod).to(DEV), self.sh.to(DEV),
            self.sc.to(DEV), (self.gt if gate is None else gate).to(DEV), *self.q1, *self.q2, self.ws,
            self.bytes, out)
        st = self.h3.h3_sync_status()
        _intact(self.guard, *([] if gout is None else [gout]))
        return out, st

    def stored(self):
        """y and h as the call stored them."""
        off = (self.L * self.d * 2 + 255) // 256 * 256
        y = self.ws[: self.L * self.d * 2].view(torch.bfloat16).view(self.L, self.d)
        h = self.ws[off: off + self.L * self.hidden * 2].view(torch.bfloat16).view(self.L, self.hidden)
        return to64(y), to64(h)


SHAPES = [(1, 256, 1024), (2, 256, 1024), (3, 256, 1024), (5, 128, 384), (13, 640, 1152),
          (16, 256, 1024), (17, 256, 1024), (32, 384, 640), (33, 256, 1024), (40, 256, 1024),
          (48, 128, 2048), (49, 256, 512), (64, 256, 8192), (65, 256, 1024), (130, 384, 896),
          (1, 128, 16384), (2, 128, 8192), (12, 2048, 8192), (300, 512, 2048)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("L,d,hidden", SHAPES)
def test_mlp_fp4_against_oracle_at_every_row_count(h3, fmt, L, d, hidden):
    m = _Mlp(h3, fmt, L, d, hidden)
    out, st = m.run()
    assert st == 0
    y, h = m.stored()
    mod = m.mod.numpy()
    x64, s64, c64, g64 = to64(m.x), to64(m.sh), to64(m.sc), to64(m.gt)
    what = f"fp4 mlp {fmt} {L}x{d}x{hidden}"
    assert_parity(y, orc.adaln_modulate(x64, mod, s64, c64), what + " y")
    h_ref = orc.gelu_tanh(orc.linear(f4.dequant(y, fmt), f4.dequant(to64(m.w1), fmt)))
    assert_parity(h, h_ref, what + " h")
    branch = orc.linear(f4.dequant(h, fmt), f4.dequant(to64(m.w2), fmt))
    assert_parity(to64(out), orc.gated_residual(x64, branch, mod, g64), what + " out")
    exact = orc.mlp_block(x64, mod, s64, c64, g64, to64(m.w1), to64(m.w2))
    assert_parity(to64(out), exact["out"], what + " out vs exact", max_rel_rms=FP4_MAX,
                  mean_rel=FP4_MEAN)
    # in place, and the same bits again
    xin = m.x.to(DEV)
    got, st = m.run(x=xin, out=xin)
    assert st == 0 and torch.equal(got, out)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("L,hidden", [(1, 512), (2, 512), (3, 512), (16, 512), (40, 512), (64, 8192), (70, 512)])
def test_zero_gate_returns_the_input_at_every_row_count(h3, fmt, L, hidden):
    m = _Mlp(h3, fmt, L, 256, hidden)
    out, st = m.run(gate=torch.zeros(3, 256))
    assert st == 0 and torch.equal(out.cpu(), m.x)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("L,hidden", [(1, 512), (2, 512), (3, 512), (16, 512), (40, 512), (64, 8192), (70, 512)])
def test_a_bad_modality_is_reported_at_every_row_count(h3, fmt, L, hidden):
    m = _Mlp(h3, fmt, L, 256, hidden)
    good, st = m.run()
    assert st == 0
    for row in sorted({0, L // 2, L - 1}):
        mod = m.mod.clone()
        mod[row] = 3 if row else 255
        out, st = m.run(mod=mod)
        assert st == 5
        nan = torch.isnan(out).cpu()
        assert bool(nan[row].all()) and int(nan.any(dim=1).sum()) == 1
        keep = torch.arange(L) != row
        assert torch.equal(out.cpu()[keep], good.cpu()[keep])
        assert m.run()[1] == 0      # reported once
