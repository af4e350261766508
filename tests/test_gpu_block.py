"""The operators together: a pre-norm block trained end to end, and the layer's two new hooks."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
import oracle
from mixture_experts_layer_14_gb300 import train_block
from mixture_experts_layer_14_gb300.synthetic import WORKLOADS, LayerShape, make_layer
from tests._helpers import assert_close, dims_of, ensure_lib, f64, to_dev

pytestmark = pytest.mark.gpu

MX = LayerShape("mx", 200, 256, 16, 4, 256, 256, 1, 0.0, "normal0.1", "mxfp8", True, 41)


def _layer(shape, dtype):
    L = to_dev(make_layer(shape, "cpu", with_dy=True))
    D = dims_of(shape, dtype=dtype)
    L["prepared"], L["prepared_bwd"] = mok.prepare_weights(D, L), mok.prepare_weights_bwd(D, L)
    ws = torch.zeros(mok.workspace_size(D), dtype=torch.uint8, device="cuda")
    idx, w, logits = mok.route(D, L["x"], L["W_router"], L["bias"], ws, want_logits=True)
    return D, L, ws, mok.dispatch_index(D, idx, w, ws), logits


def test_forward_from_given_codes():
    """The codes that the layer's own quantiser would make give its bits; the norm's give the same
    output up to the codes that differ because the norm rounds once."""
    ensure_lib()
    D, L, ws, routing, _ = _layer(MX, mok.MOK_MXFP8)
    want = mok.moe_forward(D, L, L["x"], routing, ws)
    q, sc = mok.mx_quantize_rows(L["x"])
    rows = torch.zeros((256, MX.d // 32), dtype=torch.uint8, device="cuda")
    rows[:MX.T] = sc
    atoms = rows.view(2, 4, 32, MX.d // 128, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    got = mok.moe_forward(D, L, L["x"], routing, ws, x_mx=(q, atoms))
    assert torch.equal(got, want)
    with pytest.raises(ValueError):
        mok.moe_forward(D, L, L["x"], routing, ws, x_mx=(q, sc))


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_backward_with_a_gradient_of_the_logits(dtype):
    """dlogits grows by it, dX by its product with W_router^T, dW_router by x^T times it; zeros and
    None give the same bits."""
    ensure_lib()
    code = mok.MOK_MXFP8 if dtype == "mxfp8" else mok.MOK_BF16
    D, L, ws, routing, logits = _layer(MX.with_(dtype=dtype), code)
    saved = torch.empty(mok.saved_size(D), dtype=torch.uint8, device="cuda")
    mok.moe_forward(D, L, L["x"], routing, ws, saved=saved)
    bws = torch.zeros(mok.workspace_size(D, backward=True), dtype=torch.uint8, device="cuda")
    aux = 0.5 * torch.randn((MX.T, MX.E), generator=torch.Generator().manual_seed(0)).cuda()
    base = mok.moe_backward(D, L, L["x"], L["dY"], saved, routing, bws)
    zero = mok.moe_backward(D, L, L["x"], L["dY"], saved, routing, bws, dlogits_aux=torch.zeros_like(aux))
    assert all(torch.equal(base[k], zero[k]) for k in base)
    got = mok.moe_backward(D, L, L["x"], L["dY"], saved, routing, bws, dlogits_aux=aux)
    assert torch.equal(got["dlogits"], base["dlogits"] + aux)
    for k in ("dW_gate", "dW_up", "dW_down", "dWs_gate", "dWs_up", "dWs_down"):
        assert torch.equal(got[k], base[k])
    total = f64(got["dlogits"])
    assert_close("dW_router", f64(got["dW_router"]), f64(L["x"]).T @ total)
    # dX's bf16 rounding is relative to dX, the router's share a part of it
    want = f64(base["dX"]) + f64(aux) @ f64(L["W_router"]).T
    assert_close("dX", f64(got["dX"]), want)


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
def test_block_forward_and_backward(dtype, res):
    """The block equals its parts, called one by one."""
    ensure_lib()
    shape = MX.with_(dtype=dtype)
    D = dims_of(shape, dtype=mok.MOK_MXFP8 if dtype == "mxfp8" else mok.MOK_BF16)
    W = to_dev(make_layer(shape, "cpu", with_dy=True))
    x, dY = W.pop("x"), W.pop("dY")
    W["norm"] = torch.linspace(0.5, 1.5, shape.d, device="cuda")
    r = None if res is None else (3 * torch.randn(x.shape, generator=torch.Generator().manual_seed(1))).to(res).cuda()
    dh = None if r is None else torch.randn(x.shape, generator=torch.Generator().manual_seed(2)).to(res).cuda()
    b = mok.MoEBlock(D, W, alpha=0.1, z_coef=1e-2)
    offsets = torch.tensor([0, 50, 50, 200], dtype=torch.int32, device="cuda")
    y, h = b.forward(x, r, training=True, seq_offsets=offsets)
    n = mok.rms_norm(x, W["norm"], residual=r)
    assert torch.equal(b.u, n["y"]) and torch.equal(h, n.get("residual", x))
    g = b.backward(dY, dh)
    routing = b.layer.routing
    parts = mok.moe_backward(D, W, n["y"], dY, b.layer.saved, routing,
                             torch.zeros(mok.workspace_size(D, backward=True), dtype=torch.uint8, device="cuda"),
                             dlogits_aux=b.aux["dlogits"])
    want = mok.rms_norm_backward(parts["dX"], h, W["norm"], dres=dh)
    assert torch.equal(g["dinput"], want["dx"]) and torch.equal(g["norm"], want["dweight"])
    assert torch.equal(g["dW_router"], parts["dW_router"])
    names, params = b.parameters()
    assert all(p.shape == q.shape for p, q in zip(params, b.gradients(g)))
    counts = torch.bincount(routing["topk_idx"].flatten().long(), minlength=shape.E)
    assert torch.equal(b.aux["counts"].sum(0), counts.to(torch.int32))
    if dtype == "bf16":
        sh = (f64(W["Ws_gate"]), f64(W["Ws_up"]), f64(W["Ws_down"]))
        logits = oracle.router_logits(f64(n["y"]), f64(W["W_router"]), f64(W["bias"]))
        idx = routing["topk_idx"].cpu().numpy()
        assert_close("y", f64(y), oracle.moe_forward(f64(n["y"]), f64(W["W_gate"]), f64(W["W_up"]), f64(W["W_down"]), sh,
                                                     idx, oracle.weights_for_selection(logits, idx)))


def test_block_without_a_shared_expert():
    ensure_lib()
    shape = MX.with_(dtype="bf16", n_shared=0, F_shared=0)
    D = dims_of(shape)
    W = to_dev(make_layer(shape, "cpu", with_dy=True))
    x, dY = W.pop("x"), W.pop("dY")
    W["norm"] = torch.ones(shape.d, dtype=torch.bfloat16, device="cuda")
    b = mok.MoEBlock(D, W, alpha=0.1)
    with pytest.raises(RuntimeError):
        b.backward(dY)
    b.forward(x, training=True)
    names, params = b.parameters()
    grads = b.gradients(b.backward(dY))
    assert names == ["W_router", "W_gate", "W_up", "W_down", "norm"]
    assert all(p.shape == q.shape and q.isfinite().all() for p, q in zip(params, grads))
    mok.AdamW(params).step(grads, 1e-3, clip=mok.grad_norm(grads, 1.0))
    assert b.forward(x)[0].isfinite().all()


@pytest.mark.parametrize("dtype,states", [("bf16", "f32"), ("bf16", "mxfp8"), ("mxfp8", "f32"), ("mxfp8", "mxfp8")])
def test_training_reduces_the_error(dtype, states):
    ensure_lib()
    e = train_block.train(steps=30, dtype=dtype, states=states)
    assert np.isfinite(e).all() and e[-1] < 0.5 * e[0], e


def test_tiny_workload_block_is_reproducible():
    ensure_lib()
    shape = WORKLOADS["tiny"]
    runs = [train_block.train(steps=5, T=shape.T, d=shape.d, E=shape.E, k=shape.k, F=128) for _ in range(2)]
    assert runs[0] == runs[1]
