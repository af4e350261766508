"""Selection and balance loss together on tokens without open experts: of -inf logits they have no gradient
at all; of a type's lowest value they are tokens of the balance loss unless its mask leaves them out."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests._helpers import ensure_lib

pytestmark = pytest.mark.gpu

LOWEST = float(torch.finfo(torch.float32).min)


def _run(l, sel, mask=None):
    T, E = l.shape
    D, ws = mok.dims(T, 128, E, 4, 128, 0, 0), torch.zeros(256, dtype=torch.uint8, device="cuda")
    bws = torch.zeros(mok.balance_loss_workspace_size(D, 1), dtype=torch.uint8, device="cuda")
    idx, w = mok.select_experts(D, sel, l, ws, bias=torch.zeros(E, device="cuda"))
    aux = mok.balance_loss(D, l, idx, bws, 0.02, z_coef=1e-4, token_mask=mask)
    dl = mok.select_experts_backward(D, sel, l, idx, torch.ones_like(w), ws, dlogits_aux=aux["dlogits"])
    assert mok.read_status(ws) == 0 and mok.read_status(bws) == 0
    return w, aux, dl


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("value,masked", [(-np.inf, False), (-np.inf, True), (LOWEST, True)])
def test_tokens_without_open_experts(scoring, renorm, value, masked):
    ensure_lib()
    l = torch.randn((70, 32), generator=torch.Generator().manual_seed(2)).cuda()
    l[:, 5] = value                       # one expert shut off for all
    mask = torch.ones(70, dtype=torch.bool, device="cuda")
    mask[[3, 40]] = not masked
    sel = mok.Selection(scoring, renormalise=renorm)
    shut = l.clone()
    shut[[3, 40]] = value
    w, aux, dl = _run(shut, sel, mask)
    assert not w[[3, 40]].any() and not aux["dlogits"][[3, 40]].any() and not dl[[3, 40]].any()
    assert torch.isfinite(aux["loss"]).all() and torch.isfinite(dl).all() and not dl[:, 5].any()
    assert dl[[0, 69]].any()


def test_lowest_value_without_a_mask_is_a_token():
    """As mok.h says: a uniform row, whose z loss is the square of its log-sum-exp."""
    ensure_lib()
    l = torch.randn((70, 32), generator=torch.Generator().manual_seed(2)).cuda()
    l[3] = LOWEST
    w, aux, dl = _run(l, mok.Selection("sigmoid"))
    assert not w[3].any() and torch.isinf(aux["loss"][1]) and torch.isfinite(aux["loss"][0])
    assert torch.equal(dl[3], aux["dlogits"][3]) and (dl[3] < -1e30).all()
    others = [t for t in range(70) if t != 3]
    assert torch.isfinite(dl[others]).all() and dl[others].abs().max() < 10
