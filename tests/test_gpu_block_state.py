"""What a block and a layer keep between their forward and backward passes."""

import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from mixture_experts_layer_14_gb300.synthetic import LayerShape, make_layer
from tests._helpers import dims_of, ensure_lib, to_dev

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
