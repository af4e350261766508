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


def test_route_for_logits_alone():
    D = mok.dims(16, 128, 16, 4, 128, 0, 0)

    def call(idx, w, logits, n=16):
        return ensure_lib().mok_route(ctypes.byref(D), P, P, NULL, idx, w, logits, P, n, NULL)
    assert call(NULL, NULL, NULL) == INVALID and call(P, NULL, P) == INVALID and call(NULL, P, P) == INVALID
    assert call(NULL, NULL, P) == WORKSPACE  # as far as the size of the workspace


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


def _args(**kw):
    a = dict(eps=1e-6, res_scale=1.0, res_type=0, post_type=0, gate_type=0, weight_type=0, post_weight=P, gate=NULL,
             token_gate=NULL, weight=P)
    a.update({k: v for k, v in kw.items() if k in a})
    return mok.Sandwich(**a), {k: v for k, v in kw.items() if k not in a}


def _sandwich(T=4, d=256, null=False, **kw):
    a, kw = _args(**kw)
    p = dict(x=P, r=P, ro=P, y=P, q=NULL, sc=NULL, layout=0, xq=NULL, xs=NULL, hq=NULL, hs=NULL)
    p.update(kw)
    return ensure_lib().mok_sandwich_norm(None if null else ctypes.byref(a), T, d, *p.values(), NULL)


PARAMS = [(dict(null=True), INVALID), (dict(T=-1), UNSUPPORTED), (dict(d=0), UNSUPPORTED), (dict(d=12), UNSUPPORTED),
          (dict(d=32776), UNSUPPORTED), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
          (dict(res_scale=float("inf")), INVALID), (dict(res_type=2), INVALID), (dict(post_type=-1), INVALID),
          (dict(gate_type=2), INVALID), (dict(weight_type=3), INVALID), (dict(post_weight=NULL), INVALID),
          (dict(post_weight=ODD), UNSUPPORTED), (dict(weight=ODD), UNSUPPORTED)]


@pytest.mark.parametrize("kw,rc", PARAMS + [
    (dict(gate=ODD), UNSUPPORTED), (dict(token_gate=ODD4), UNSUPPORTED),
    (dict(d=64, q=P, sc=P), UNSUPPORTED), (dict(d=64, xq=P, xs=P, hq=P, hs=P), UNSUPPORTED), (dict(x=NULL), INVALID),
    (dict(r=NULL), INVALID), (dict(ro=NULL), INVALID), (dict(y=NULL), INVALID), (dict(weight=NULL), INVALID),
    (dict(weight=NULL, y=NULL, q=P, sc=P), INVALID), (dict(q=P), INVALID), (dict(sc=P), INVALID), (dict(layout=2), INVALID),
    (dict(xq=P), INVALID), (dict(xq=P, xs=P, hq=P), INVALID), (dict(x=ODD), UNSUPPORTED), (dict(ro=ODD), UNSUPPORTED),
    (dict(y=ODD), UNSUPPORTED), (dict(q=P, sc=ODD), UNSUPPORTED), (dict(xq=P, xs=P, hq=ODD, hs=P), UNSUPPORTED)])
def test_sandwich_norm(kw, rc):
    assert _sandwich(**kw) == rc


def _sandwich_bwd(T=4, d=256, null=False, n=1 << 30, **kw):
    a, kw = _args(**kw)
    p = dict(dy=P, dres=P, x=P, xs=NULL, h=P, hs=NULL, dx=P, dr=P, dpost=P, dgate=NULL, dtg=NULL, dw=P, ws=P)
    p.update(kw)
    return ensure_lib().mok_sandwich_norm_backward(None if null else ctypes.byref(a), T, d, *p.values(), n, NULL)


@pytest.mark.parametrize("kw,rc", PARAMS + [
    (dict(gate=ODD, dgate=P), UNSUPPORTED), (dict(token_gate=ODD4, dtg=P), UNSUPPORTED), (dict(token_gate=P, dtg=ODD4), UNSUPPORTED),
    (dict(gate=P), INVALID), (dict(dgate=P), INVALID), (dict(token_gate=P), INVALID), (dict(dtg=P), INVALID),
    (dict(weight=NULL), INVALID), (dict(weight=NULL, dw=NULL), INVALID), (dict(dw=NULL), INVALID), (dict(dy=NULL), INVALID),
    (dict(h=NULL), INVALID), (dict(x=NULL), INVALID), (dict(dx=NULL), INVALID), (dict(dr=NULL), INVALID),
    (dict(dpost=NULL), INVALID), (dict(ws=NULL), INVALID), (dict(dy=NULL, weight=NULL, dw=NULL, dres=NULL), INVALID),
    (dict(xs=P), INVALID), (dict(hs=P), INVALID), (dict(d=64, xs=P, hs=P), UNSUPPORTED), (dict(dres=ODD), UNSUPPORTED),
    (dict(xs=ODD, hs=P), UNSUPPORTED), (dict(dx=ODD), UNSUPPORTED), (dict(dpost=ODD), UNSUPPORTED), (dict(n=64), WORKSPACE)])
def test_sandwich_norm_backward(kw, rc):
    assert _sandwich_bwd(**kw) == rc


def test_sandwich_binding():
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256)
    c = (torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 8, dtype=torch.uint8))
    assert ensure_lib().mok_sandwich_norm_workspace_size(4, 12) == 0
    assert mok.sandwich_norm_workspace_size(4, 256) >= 256 + 8 * 256
    for bad in (dict(x=x[0]), dict(x=x.float()), dict(residual=x[:2]), dict(residual=x.half()), dict(post_weight=w[1:]),
                dict(weight=w.double()), dict(gate=w[:3]), dict(token_gate=w), dict(mx="rows", weight=None), dict(mx="cols"),
                dict(save="int8"), dict()):                                   # the last: not on a GPU
        with pytest.raises(ValueError):
            mok.sandwich_norm(**dict(dict(x=x, residual=x, post_weight=w, weight=w), **bad))
    for bad in (dict(dy=None), dict(weight=None), dict(h=None), dict(dy=None, weight=None), dict(x=c), dict(h=c),
                dict(residual_dtype=torch.float32), dict(dres=x.float()), dict(x=(c[0], c[1][:2]), h=c), dict(x=c, h=c,
                residual_dtype=torch.float16), dict(x=x[0]), dict()):
        with pytest.raises(ValueError):
            mok.sandwich_norm_backward(**dict(dict(x=x, h=x, post_weight=w, dy=x, weight=w), **bad))


def _pack(rows=4, K=64, src=P, kind=0, q=P, s=P):
    return ensure_lib().mok_activation_pack(rows, K, src, kind, q, s, NULL)


def _unpack(rows=4, K=64, src=P, kind=0, q=P, s=P, layout=0):
    return ensure_lib().mok_activation_unpack(rows, K, q, s, layout, src, kind, NULL)


@pytest.mark.parametrize("kw,rc", [
    (dict(rows=-1), UNSUPPORTED), (dict(K=0), UNSUPPORTED), (dict(K=48), UNSUPPORTED), (dict(rows=1 << 36), UNSUPPORTED),
    (dict(kind=2), INVALID), (dict(src=NULL), INVALID), (dict(q=NULL), INVALID), (dict(s=NULL), INVALID),
    (dict(src=ODD), UNSUPPORTED), (dict(q=ODD), UNSUPPORTED), (dict(s=ODD), UNSUPPORTED)])
def test_activation_pack(kw, rc):
    assert _pack(**kw) == rc and _unpack(**kw) == rc


def test_activation_unpack_layouts_and_saved():
    L = ensure_lib()
    assert _unpack(layout=2) == INVALID and _unpack(layout=1) == UNSUPPORTED
    assert _pack(rows=0, src=NULL, q=NULL, s=NULL) == 0 and _unpack(rows=0, src=NULL, q=NULL, s=NULL) == 0
    D, D4 = mok.dims(16, 256, 8, 2, 256, 256, 1), mok.dims(16, 256, 8, 2, 256, 256, 1, mok.MOK_NVFP4)
    D8, D0 = mok.dims(16, 256, 8, 2, 256, 256, 1, mok.MOK_MXFP8), mok.dims(0, 256, 8, 2, 256, 256, 1)
    n = 2 * (32 + 16) * 256
    assert n * 33 // 32 <= L.mok_packed_saved_size(ctypes.byref(D)) <= n * 33 // 32 + 8 * 1024
    assert L.mok_packed_saved_size(ctypes.byref(D4)) == 0

    def pack(d, saved=P, packed=P):
        return L.mok_saved_pack(ctypes.byref(d), saved, packed, NULL)

    def unpack(d, packed=P, x=P, inv=P, saved=P):
        return L.mok_saved_unpack(ctypes.byref(d), packed, x, inv, saved, NULL)
    assert pack(D4) == UNSUPPORTED and unpack(D4) == UNSUPPORTED
    assert pack(D, saved=NULL) == INVALID and pack(D, packed=NULL) == INVALID and pack(D, saved=ODD) == UNSUPPORTED
    assert unpack(D, packed=NULL) == INVALID and unpack(D, x=NULL) == INVALID and unpack(D, inv=NULL) == INVALID
    assert unpack(D8, saved=NULL) == INVALID and unpack(D, x=ODD) == UNSUPPORTED and unpack(D, packed=ODD) == UNSUPPORTED
    assert pack(D0, NULL, NULL) == 0 and unpack(D0, NULL, NULL, NULL, NULL) == 0


def test_packing_binding():
    x = torch.zeros(4, 64)
    for bad in (x.half(), torch.zeros(()), torch.zeros(4, 0), x):                     # the last: not on a GPU
        with pytest.raises(ValueError):
            mok.activation_pack(bad)
    c, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    for args in ((c, s, torch.float16), (c, s, torch.float32, "columns"), (c.float(), s), (c, s[:2]), (c, s)):
        with pytest.raises(ValueError):
            mok.activation_unpack(*args)
    with pytest.raises(ValueError):
        mok.saved_pack(mok.dims(16, 256, 8, 2, 256, 256, 1), torch.zeros(8, dtype=torch.uint8))
