"""Refusals of the entry points around the layer: every wrong call is answered on the host, before
any CUDA call (no GPU needed)."""

import ctypes

import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests._helpers import ensure_lib

NULL, P, ODD = None, 0x1000, 0x1008
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


def _norm(T=4, d=256, eps=1e-6, x=P, r=NULL, rt=0, w=P, wt=0, y=P, ro=NULL, q=NULL, sc=NULL, layout=0):
    return ensure_lib().mok_rms_norm(T, d, eps, x, r, rt, w, wt, y, ro, q, sc, layout, NULL)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), UNSUPPORTED), (dict(d=0), UNSUPPORTED), (dict(d=12), UNSUPPORTED), (dict(d=32776), UNSUPPORTED),
    (dict(d=64, q=P, sc=P), UNSUPPORTED), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(rt=2), INVALID), (dict(wt=-1), INVALID), (dict(layout=2), INVALID),
    (dict(x=NULL), INVALID), (dict(w=NULL), INVALID), (dict(y=NULL), INVALID), (dict(q=P), INVALID),
    (dict(r=P), INVALID), (dict(ro=P), INVALID), (dict(x=ODD), UNSUPPORTED), (dict(w=ODD), UNSUPPORTED),
    (dict(y=ODD), UNSUPPORTED), (dict(r=ODD, ro=P), UNSUPPORTED), (dict(r=P, ro=ODD), UNSUPPORTED),
    (dict(q=ODD, sc=P), UNSUPPORTED), (dict(q=P, sc=ODD), UNSUPPORTED)])
def test_rms_norm(kw, rc):
    assert _norm(**kw) == rc


def _norm_bwd(T=4, d=256, eps=1e-6, dy=P, s=P, rt=0, w=P, wt=0, dres=NULL, dx=P, dr=NULL, dw=P, ws=P, n=1 << 30):
    return ensure_lib().mok_rms_norm_backward(T, d, eps, dy, s, rt, w, wt, dres, dx, dr, dw, ws, n, NULL)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), UNSUPPORTED), (dict(d=4), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(rt=7), INVALID),
    (dict(wt=7), INVALID), (dict(dy=NULL), INVALID), (dict(s=NULL), INVALID), (dict(w=NULL), INVALID),
    (dict(dx=NULL), INVALID), (dict(dw=NULL), INVALID), (dict(ws=NULL), INVALID), (dict(dy=ODD), UNSUPPORTED),
    (dict(dres=ODD), UNSUPPORTED), (dict(dw=ODD), UNSUPPORTED), (dict(ws=ODD), UNSUPPORTED), (dict(n=100), WORKSPACE)])
def test_rms_norm_backward(kw, rc):
    assert _norm_bwd(**kw) == rc


def _balance(D=None, logits=P, idx=P, off=NULL, S=1, mask=NULL, alpha=0.1, z=0.0, grad=NULL, counts=P, loss=P, dl=P,
             ws=P, n=1 << 30):
    D = D or mok.dims(16, 128, 8, 2, 128, 0, 0)
    return ensure_lib().mok_balance_loss(ctypes.byref(D), logits, idx, off, S, mask, alpha, z, grad, counts, loss, dl,
                                         ws, n, NULL)


@pytest.mark.parametrize("kw,rc", [
    (dict(D=mok.dims(16, 128, 12, 2, 128, 0, 0)), UNSUPPORTED), (dict(D=mok.dims(-1, 128, 8, 2, 128, 0, 0)), UNSUPPORTED),
    (dict(S=0, off=P), INVALID), (dict(S=2), INVALID), (dict(S=1 << 30, off=P), UNSUPPORTED),
    (dict(alpha=float("nan")), INVALID), (dict(z=float("inf")), INVALID), (dict(logits=NULL), INVALID),
    (dict(idx=NULL), INVALID), (dict(counts=NULL), INVALID), (dict(loss=NULL), INVALID), (dict(ws=NULL), INVALID),
    (dict(logits=ODD), UNSUPPORTED), (dict(counts=ODD), UNSUPPORTED), (dict(dl=ODD), UNSUPPORTED),
    (dict(ws=ODD), UNSUPPORTED), (dict(n=64), WORKSPACE), (dict(idx=0x1002), UNSUPPORTED), (dict(loss=0x1001), UNSUPPORTED),
    (dict(off=0x1002), UNSUPPORTED), (dict(grad=0x1002), UNSUPPORTED)])
def test_balance_loss(kw, rc):
    assert _balance(**kw) == rc


def _norm_of(n=1, grads=(P,), numel=(100,), types=(0,), limit=1.0, out=P, ws=P, size=1 << 20):
    a = (ctypes.c_void_p * len(grads))(*grads) if grads is not None else None
    b = (ctypes.c_int64 * len(numel))(*numel) if numel is not None else None
    c = (ctypes.c_int32 * len(types))(*types) if types is not None else None
    return ensure_lib().mok_grad_norm(n, a, b, c, limit, out, ws, size, NULL)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=-1), INVALID), (dict(grads=None), INVALID), (dict(numel=None), INVALID), (dict(types=None), INVALID),
    (dict(out=NULL), INVALID), (dict(ws=NULL), INVALID), (dict(limit=float("nan")), INVALID), (dict(grads=(None,)), INVALID),
    (dict(numel=(-1,)), INVALID), (dict(types=(2,)), INVALID), (dict(grads=(ODD,)), UNSUPPORTED), (dict(ws=ODD), UNSUPPORTED),
    (dict(numel=(1 << 41,)), UNSUPPORTED), (dict(size=128), WORKSPACE), (dict(out=0x1002), UNSUPPORTED)])
def test_grad_norm(kw, rc):
    assert _norm_of(**kw) == rc


def _adam(args=None, n=1, **kw):
    a = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1, state_format=0)
    a.update(args or {})
    t = dict(param=P, grad=P, master=P, exp_avg=P, exp_avg_sq=P, exp_avg_scale=NULL, exp_avg_sq_scale=NULL, numel=100,
             weight_decay=0.0, param_type=0, grad_type=0)
    t.update(kw)
    table = (mok.AdamWTensor * 1)(mok.AdamWTensor(**t))
    return ensure_lib().mok_adamw_step(ctypes.byref(mok.AdamWArgs(**a)), table, n, NULL, NULL)


@pytest.mark.parametrize("args", [dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")),
                                  dict(eps=0.0), dict(eps=float("inf")), dict(lr=float("nan")), dict(step=0),
                                  dict(state_format=2)])
def test_adamw_args(args):
    assert _adam(args) == INVALID


@pytest.mark.parametrize("kw,rc", [
    (dict(param=NULL), INVALID), (dict(grad=NULL), INVALID), (dict(exp_avg=NULL), INVALID), (dict(exp_avg_sq=NULL), INVALID),
    (dict(master=NULL), INVALID), (dict(param_type=1), INVALID), (dict(param_type=2), INVALID), (dict(grad_type=-1), INVALID),
    (dict(numel=-5), INVALID), (dict(weight_decay=float("inf")), INVALID), (dict(param=ODD), UNSUPPORTED),
    (dict(grad=ODD), UNSUPPORTED), (dict(master=ODD), UNSUPPORTED), (dict(exp_avg=ODD), UNSUPPORTED),
    (dict(numel=1 << 41), UNSUPPORTED), (dict(n=-1), INVALID), (dict(args=dict(state_format=1)), INVALID)])
def test_adamw_tensor(kw, rc):
    assert _adam(**kw) == rc


def test_nothing_to_do_is_fine():
    L = ensure_lib()
    assert _norm(T=0, x=NULL, w=NULL, y=NULL) == 0
    assert L.mok_adamw_step(ctypes.byref(mok.AdamWArgs(1e-3, 0.9, 0.95, 1e-8, 1, 0)), None, 0, None, None) == 0
    assert _adam(numel=0, param=NULL, grad=NULL) == 0


def test_forward_from_codes_and_sizes():
    L = ensure_lib()
    D, W = mok.dims(16, 256, 8, 2, 256, 0, 0), mok.Weights()
    rest = [P] * 8 + [NULL, P, 1 << 40, NULL]
    assert L.mok_moe_forward_mx(ctypes.byref(D), ctypes.byref(W), *([P] * 8 + [NULL, P, 1 << 40, NULL])) == UNSUPPORTED
    D8 = mok.dims(16, 256, 8, 2, 256, 0, 0, mok.MOK_MXFP8)
    assert L.mok_moe_forward_mx(ctypes.byref(D8), ctypes.byref(W), NULL, *rest[1:]) == INVALID
    assert L.mok_moe_forward_mx(ctypes.byref(D8), ctypes.byref(W), P, NULL, *rest[2:]) == INVALID
    assert L.mok_rms_norm_workspace_size(100, 12) == 0 and L.mok_rms_norm_workspace_size(100, 256) >= 256
    assert L.mok_balance_loss_workspace_size(ctypes.byref(D), 0) == 0
    assert mok.balance_loss_workspace_size(D, 5) > 256
    assert L.mok_grad_norm_workspace_size(1, (ctypes.c_int64 * 1)(-1)) == 0


def test_binding_checks():
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256)
    for bad in (dict(x=x.float()), dict(x=x[0]), dict(weight=w[:-1]), dict(weight=w.double()), dict(mx="columns"),
                dict(residual=x[:2]), dict(x=x)):                          # the last: not on a GPU
        with pytest.raises(ValueError):
            mok.rms_norm(**dict(dict(x=x, weight=w), **bad))
    with pytest.raises(ValueError):
        mok.rms_norm_backward(x, x.half(), w)
    with pytest.raises(ValueError):
        mok.TensorList([x])
    with pytest.raises(ValueError):
        mok.TensorList([x.half()])
    with pytest.raises(ValueError):
        mok.AdamW([], states="int4")
    with pytest.raises(ValueError):
        mok._want_ws(torch.zeros(8, dtype=torch.uint8), torch.device("cpu"))
    with pytest.raises(ValueError):
        mok._want_ws(torch.zeros(8), torch.device("cpu"))
    D = mok.dims(4, 128, 8, 2, 128, 0, 0)
    with pytest.raises(ValueError):
        mok.balance_loss(D, torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64), torch.zeros(8), 0.1)
