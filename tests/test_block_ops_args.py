"""Refusals of the block's operators: every wrong call is answered on the host, before any CUDA call
(no GPU needed)."""

import ctypes

import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests._helpers import ensure_lib

NULL, P, ODD, ODD4 = None, 0x1000, 0x1008, 0x1002
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


def _sel(**kw):
    s = mok.Selection()
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _select(D=None, sel=None, logits=P, bias=NULL, idx=P, w=P, ws=P, n=1 << 20, null_sel=False):
    D = D or mok.dims(16, 128, 16, 4, 128, 0, 0)
    sel = None if null_sel else ctypes.byref(sel or _sel())
    return ensure_lib().mok_select_experts(ctypes.byref(D), sel, logits, bias, idx, w, ws, n, NULL)


def _select_bwd(D=None, sel=None, logits=P, idx=P, dw=P, aux=NULL, dl=P, ws=P, n=1 << 20):
    D = D or mok.dims(16, 128, 16, 4, 128, 0, 0)
    return ensure_lib().mok_select_experts_backward(ctypes.byref(D), ctypes.byref(sel or _sel()), logits, idx, dw, aux,
                                                    dl, ws, n, NULL)


SELECTIONS = [(dict(score=2), INVALID), (dict(score=-1), INVALID), (dict(group_score=2), INVALID),
              (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(n_groups=0), UNSUPPORTED),
              (dict(n_groups=3), UNSUPPORTED), (dict(n_groups=64), UNSUPPORTED), (dict(topk_groups=0), UNSUPPORTED),
              (dict(topk_groups=2), UNSUPPORTED), (dict(n_groups=8, topk_groups=1), UNSUPPORTED)]  # the last: k = 4 of 2


@pytest.mark.parametrize("kw,rc", SELECTIONS)
def test_selection(kw, rc):
    assert _select(sel=_sel(**kw)) == rc
    assert _select_bwd(sel=_sel(**kw)) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(D=mok.dims(16, 128, 12, 2, 128, 0, 0)), UNSUPPORTED), (dict(D=mok.dims(-1, 128, 8, 2, 128, 0, 0)), UNSUPPORTED),
    (dict(logits=NULL), INVALID), (dict(idx=NULL), INVALID), (dict(w=NULL), INVALID), (dict(ws=NULL), INVALID),
    (dict(null_sel=True), INVALID), (dict(logits=ODD), UNSUPPORTED), (dict(bias=ODD), UNSUPPORTED),
    (dict(idx=ODD4), UNSUPPORTED), (dict(w=ODD4), UNSUPPORTED), (dict(ws=ODD), UNSUPPORTED), (dict(n=255), WORKSPACE)])
def test_select_experts(kw, rc):
    assert _select(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(logits=NULL), INVALID), (dict(idx=NULL), INVALID), (dict(dw=NULL), INVALID), (dict(dl=NULL), INVALID),
    (dict(ws=NULL), INVALID), (dict(logits=ODD), UNSUPPORTED), (dict(aux=ODD), UNSUPPORTED), (dict(dl=ODD), UNSUPPORTED),
    (dict(idx=ODD4), UNSUPPORTED), (dict(dw=ODD4), UNSUPPORTED), (dict(n=0), WORKSPACE)])
def test_select_experts_backward(kw, rc):
    assert _select_bwd(**kw) == rc


def test_moe_backward_select():
    D, W = mok.dims(16, 128, 16, 4, 128, 0, 0), mok.Weights()

    def call(sel, logits, dlogits=P):
        return ensure_lib().mok_moe_backward_select(ctypes.byref(D), ctypes.byref(W), P, P, P, ctypes.byref(sel), logits,
                                                    *([P] * 14), dlogits, P, P, 1 << 40, NULL)
    assert call(_sel(score=5), P) == INVALID
    assert call(_sel(n_groups=3), P) == UNSUPPORTED
    assert call(_sel(), NULL) == INVALID
    assert call(_sel(), ODD) == UNSUPPORTED
    assert call(_sel(), P, ODD) == UNSUPPORTED
    assert call(_sel(), P) == INVALID  # W is empty


def test_selection_binding():
    for bad in (dict(scoring="relu"), dict(group_score="sum")):
        with pytest.raises(ValueError):
            mok.Selection(**bad)
    D, l = mok.dims(4, 128, 8, 2, 128, 0, 0), torch.zeros(4, 8)
    for args in ((torch.zeros(4, 9), torch.zeros(256)), (l.double(), torch.zeros(256)), (l, torch.zeros(256))):
        with pytest.raises(ValueError):  # the last: not on a GPU
            mok.select_experts(D, mok.Selection(), *args)
    with pytest.raises(ValueError):
        mok.select_experts_backward(D, mok.Selection(), l, torch.zeros(4, 2), torch.zeros(4, 2), torch.zeros(256))
