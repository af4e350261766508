"""Experts whose bias is -inf: the last choice, with their score's weight (the bias ranks and does nothing
else); experts whose logit is -inf: weight 0, whatever their bias."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests import _block
from tests._helpers import ensure_lib, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("low", [-np.inf, float(np.finfo(np.float32).min), -1e30])
def test_shut_by_bias_and_by_logit(scoring, renorm, low):
    ensure_lib()
    l = np.random.default_rng(1).normal(size=(5, 16)).astype(np.float32)
    bias = np.zeros(16, dtype=np.float32)
    bias[3:] = low
    l[1:, 2], l[2:, 4] = low, low
    D, ws = mok.dims(5, 128, 16, 6, 128, 0, 0), torch.zeros(256, dtype=torch.uint8, device="cuda")
    sel = mok.Selection(scoring, renormalise=renorm, scale=2.0)
    idx, w = mok.select_experts(D, sel, torch.from_numpy(l).cuda(), ws, bias=torch.from_numpy(bias).cuda())
    idx, w = idx.cpu().numpy(), f64(w)
    for t in range(5):
        open_ = [e for e in range(3) if l[t, e] > -1e30]
        assert sorted(idx[t, :len(open_)]) == open_
        # behind them the others by index, with a weight unless their logit shuts them off
        assert idx[t, len(open_):].tolist() == [e for e in range(16) if e not in open_][:6 - len(open_)]
    assert ((w == 0) == (np.take_along_axis(l, idx, 1) <= -1e30)).all()
    s = np.take_along_axis(_block.scores(l, scoring), idx, 1)
    want = 2.0 * (s / s.sum(1, keepdims=True) if renorm else s)
    assert (np.abs(w - want) <= 2.0 ** -18 * want).all()  # as in the other tests of the weights
    assert mok.read_status(ws) == 0
