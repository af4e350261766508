"""What a block and a layer keep between their forward and backward passes, and the layer on codes
that it is given."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
import oracle
from mixture_experts_layer_14_gb300.synthetic import LayerShape, make_layer
from tests._helpers import assert_close, dims_of, ensure_lib, f64, to_dev

pytestmark = pytest.mark.gpu

MX = LayerShape("mx", 200, 256, 16, 4, 256, 256, 1, 0.0, "normal0.1", "mxfp8", True, 43)
CODE = {"bf16": mok.MOK_BF16, "mxfp8": mok.MOK_MXFP8}


def _block(dtype, **kw):
    shape = MX.with_(dtype=dtype)
    D = dims_of(shape, dtype=CODE[dtype])
    W = to_dev(make_layer(shape, "cpu", with_dy=True))
    x, dY = W.pop("x"), W.pop("dY")
    W["norm"] = torch.linspace(0.5, 1.5, shape.d, device="cuda")
    return D, W, x, dY, mok.MoEBlock(D, W, alpha=0.1, z_coef=1e-2, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_inference_between_forward_and_backward(dtype):
    """A forward that is not for training leaves the pass that backward belongs to alone."""
    ensure_lib()
    _, _, x, dY, b = _block(dtype)
    r = torch.randn(x.shape, generator=torch.Generator().manual_seed(1)).cuda()
    b.forward(x, r, training=True)
    want = b.backward(dY, r)
    y, h = b.forward(x, r, training=True)
    other_y, other_h = b.forward(x.flip(0), 3 * r)
    assert not torch.equal(other_h, h) and not torch.equal(other_y, y)
    got = b.backward(dY, r)
    assert all((want[k] is None and got[k] is None) or torch.equal(want[k], got[k]) for k in want)


def test_layer_inference_between_forward_and_backward():
    ensure_lib()
    D, W, x, dY, b = _block("bf16")
    layer = mok.MoELayer(D, W)
    layer.forward(x, training=True)
    want = layer.backward(x, dY)
    layer.forward(x, training=True)
    layer.forward(x.flip(0))
    got = layer.backward(x, dY)
    assert all((want[k] is None and got[k] is None) or torch.equal(want[k], got[k]) for k in want)


def test_a_training_forward_that_fails_leaves_nothing_to_backward():
    """The losses' arguments are refused after the layer has run: no backward of the older pass."""
    ensure_lib()
    _, _, x, dY, b = _block("bf16")
    b.forward(x, training=True)
    with pytest.raises(ValueError):
        b.forward(x, training=True, token_mask=torch.ones(3, dtype=torch.bool, device="cuda"))
    with pytest.raises(RuntimeError):
        b.backward(dY)


@pytest.mark.parametrize("missing", ["prepared", "prepared_bwd"])
def test_either_prepared_form_is_made_when_it_is_missing(missing):
    ensure_lib()
    D, W, x, dY, b = _block("mxfp8")
    b.forward(x, training=True)
    want = b.backward(dY)
    del W[missing]
    c = mok.MoEBlock(D, W, alpha=0.1, z_coef=1e-2)
    c.forward(x, training=True)
    got = c.backward(dY)
    assert torch.equal(want["dinput"], got["dinput"]) and torch.equal(want["dW_down"], got["dW_down"])


def test_weights_prepared_for_another_dtype_are_refused():
    """The NVFP4 form is smaller than the MXFP8 one: it must not reach an MXFP8 kernel."""
    ensure_lib()
    D, W, x, dY, b = _block("mxfp8")
    nv = mok.dims(D.T, D.d, D.E, D.k, D.F, D.F_shared, 1, mok.MOK_NVFP4)
    right = dict(W)
    W["prepared"] = mok.prepare_weights(nv, W)
    assert W["prepared"].numel() < right["prepared"].numel()
    with pytest.raises(ValueError):
        b.forward(x, training=True)
    W["prepared"], W["prepared_bwd"] = right["prepared"], right["prepared_bwd"][:-1]
    with pytest.raises(ValueError):
        b.forward(x, training=True)
    with pytest.raises(ValueError):
        mok.moe_forward(nv, right, x, None, b.layer.ws)


def test_forward_from_given_codes_on_a_workspace_of_its_own():
    """A zeroed workspace holds no codes of x: the output comes from the given ones."""
    ensure_lib()
    D = dims_of(MX, dtype=mok.MOK_MXFP8)
    L = to_dev(make_layer(MX, "cpu"))
    L["prepared"] = mok.prepare_weights(D, L)
    ws = torch.zeros(mok.workspace_size(D), dtype=torch.uint8, device="cuda")
    idx, w, _ = mok.route(D, L["x"], L["W_router"], L["bias"], ws)
    routing = mok.dispatch_index(D, idx, w, ws)
    want = mok.moe_forward(D, L, L["x"], routing, ws)
    q, sc = mok.mx_quantize_rows(L["x"])
    rows = torch.zeros((256, MX.d // 32), dtype=torch.uint8, device="cuda")
    rows[:MX.T] = sc
    atoms = rows.view(2, 4, 32, MX.d // 128, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    fresh = torch.zeros_like(ws)
    got = mok.moe_forward(D, L, torch.zeros_like(L["x"]), routing, fresh, x_mx=(q, atoms))
    assert torch.equal(got, want) and mok.read_status(fresh) == 0


def _oracle_forward(dtype, u, W, idx, weights):
    run = oracle.moe_forward_mxfp8 if dtype == "mxfp8" else oracle.moe_forward
    sh = (f64(W["Ws_gate"]), f64(W["Ws_up"]), f64(W["Ws_down"]))
    return run(u, f64(W["W_gate"]), f64(W["W_up"]), f64(W["W_down"]), sh, idx, weights)


@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
def test_mxfp8_block_output(res):
    """The norm's codes through the layer, against the oracle on the norm in 64 bits: the quantiser
    makes the same codes of it, but for values on a rounding boundary."""
    ensure_lib()
    D, W, x, dY, b = _block("mxfp8")
    r = None if res is None else (3 * torch.randn(x.shape, generator=torch.Generator().manual_seed(2))).to(res).cuda()
    y, _ = b.forward(x, r)
    h = f64(x) if r is None else f64(x) + f64(r)
    u = h / np.sqrt((h * h).mean(1, keepdims=True) + b.eps) * f64(W["norm"])
    idx = b.layer.routing["topk_idx"].cpu().numpy()
    logits = oracle.router_logits(f64(b.u), f64(W["W_router"]), f64(W["bias"]))
    assert_close("y", f64(y), _oracle_forward("mxfp8", u, W, idx, oracle.weights_for_selection(logits, idx)))
