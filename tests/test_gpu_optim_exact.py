"""AdamW with fp32 states: every operation rounds once.

From zero states with weights of zero the step is m = fl(om1 g), v = fl(om2 fl(g g)), w = -fl(lr
fl(m / fl(fl(sqrt v) k1 + k2))), each fl one rounding to fp32.  The same in 64 bits with a rounding to 32
after each operation gives these bits, but where the sum under the quotient, which 64 bits round
themselves first, lies within 2^-28 of a rounding boundary.
"""

import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests._helpers import ensure_lib

pytestmark = pytest.mark.gpu

BETAS, EPS, LR = (0.9, 0.95), 1e-8, 3e-3


@pytest.mark.parametrize("n", [4097, 100003])
def test_first_step_from_zero(n):
    ensure_lib()
    g = torch.randn(n, generator=torch.Generator().manual_seed(n)).mul_(1e-2).cuda()
    p = torch.zeros(n, device="cuda")
    opt = mok.AdamW([p], betas=BETAS, eps=EPS)
    opt.step([g], LR)
    fl = lambda x: x.float().double()  # noqa: E731
    c = lambda x: fl(torch.tensor(x, dtype=torch.float64, device="cuda"))  # noqa: E731
    c1, c2 = 1 / (1 - BETAS[0]), 1 / (1 - BETAS[1])
    G = g.double()
    m, v = fl(c(1 - BETAS[0]) * G), fl(c(1 - BETAS[1]) * fl(G * G))
    update = fl(m / fl(fl(v.sqrt()) * c(c2 ** 0.5 / c1) + c(EPS / c1)))
    assert torch.equal(opt.state["exp_avg"][0].double(), m) and torch.equal(opt.state["exp_avg_sq"][0].double(), v)
    want = -fl(c(LR) * update)
    assert (p.double() == want).double().mean() > 0.9999
    assert ((p.double() - want).abs() <= 2.0 ** -22 * want.abs()).all()
