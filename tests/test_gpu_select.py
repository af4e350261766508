"""Choice of experts and its gradient on the GPU against the plain 64-bit forms."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from mixture_experts_layer_14_gb300.synthetic import LayerShape, make_layer
from tests import _block
from tests._helpers import assert_close, dims_of, ensure_lib, f64, to_dev

pytestmark = pytest.mark.gpu

# Weights: expf twice and the quotient (2 ulp each), |l - m| <= 32 half ulps in the argument, sums of
# up to 512 terms in at most 21 roundings: below 64 half ulps, 2^-18 relative.  Gradients add a
# product of three such factors and one difference of dw and their mean.
W_REL = 2.0 ** -18
G_REL = 2.0 ** -16


def _ws():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def _run(l, k, bias=None, ws=None, **kw):
    ensure_lib()
    T, E = l.shape
    D = mok.dims(T, 128, E, k, 128, 0, 0)
    ws = _ws() if ws is None else ws
    sel = mok.Selection(scoring=kw["scoring"], n_groups=kw.get("groups", 1), topk_groups=kw.get("kept", 1),
                        group_score=kw.get("by", "max"), renormalise=kw.get("renorm", True), scale=kw.get("scale", 1.0))
    b = None if bias is None else torch.from_numpy(bias).cuda()
    idx, w = mok.select_experts(D, sel, torch.from_numpy(l).cuda(), ws, bias=b)
    return D, sel, idx.cpu().numpy(), w.cpu().numpy().astype(np.float64), ws


def _check(l, k, bias=None, status=0, **kw):
    _, _, idx, w, ws = _run(l, k, bias, **kw)
    ref, wref = _block.select(l, k, bias=bias, **kw)
    assert np.array_equal(idx, ref)
    assert (np.abs(w - wref) <= W_REL * wref + 1e-37).all()
    assert mok.read_status(ws) == status


def _logits(rng, T, E, masked=False):
    l = rng.normal(size=(T, E)).astype(np.float32)
    if masked:
        l[rng.random((T, E)) < 0.3] = -np.inf
        l[::7] = -np.inf
        l[3 % T] = np.finfo(np.float32).min
    return l


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,kept,by", [
    (8, 1, 1, 1, "max"), (8, 8, 1, 1, "max"), (16, 3, 16, 5, "max"), (256, 8, 8, 4, "top2"), (256, 8, 8, 1, "max"),
    (384, 8, 1, 1, "max"), (512, 8, 1, 1, "max"), (512, 7, 32, 9, "top2"), (24, 4, 3, 2, "top2"), (40, 2, 5, 1, "top2"),
    (504, 8, 9, 7, "max"), (504, 6, 21, 20, "top2"), (8, 2, 8, 2, "top2"), (160, 6, 8, 3, "max"), (136, 5, 17, 3, "top2")])
def test_against_plain(scoring, E, k, groups, kept, by):
    rng = np.random.default_rng(E + k)
    for T, masked in ((1, False), (65, False), (33, True)):
        l = _logits(rng, T, E, masked)
        bias = (rng.integers(-50, 51, E) * 1e-3).astype(np.float32)
        for b in (None, bias):
            for renorm in (True, False):
                _check(l, k, b, scoring=scoring, groups=groups, kept=kept, by=by, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept,by", [(1, 1, "max"), (8, 3, "top2"), (8, 3, "max")])
def test_keys_that_fp32_cannot_tell_apart(scoring, groups, kept, by):
    """Logits a few units in the last place from each other (no two groups' sums of two are equal
    where one stays and one goes), with biases that are equal, or that make up for the difference
    of two scores to within a rounding."""
    rng = np.random.default_rng(7)
    T, E, k = 96, 256, 8
    one = np.float32(1.0).view(np.int32)
    units = np.stack([rng.choice(4096, E, replace=False) for _ in range(T)])
    l = (one + units).astype(np.int32).view(np.float32)
    flat = np.zeros(E, dtype=np.float32)
    _check(l, k, flat, scoring=scoring, groups=groups, kept=kept, by=by)
    _check(l, k, None, scoring=scoring, groups=groups, kept=kept, by=by)
    _check(l, k, np.full(E, 0.25, dtype=np.float32), scoring=scoring, groups=groups, kept=kept, by=by)
    v = rng.normal(size=E).astype(np.float32)  # every token the same logits; bias levels the scores
    level = (0.9 - _block.scores(v, scoring)).astype(np.float32)
    l = np.tile(v, (T, 1))
    _check(l, k, level, scoring=scoring, groups=groups, kept=kept, by=by)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [None, 0.0, -0.5])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
def test_equal_numbers_go_to_the_lower_index(scoring, bias, groups, kept):
    T, E, k = 9, 64, 8
    l = np.zeros((T, E), dtype=np.float32)
    l[1] = -0.0
    l[2, ::2] = -0.0
    l[3, 40:] = 1.0
    l[4, 5:9] = -1.0
    l[5, ::3] = 2.0
    l[6] = 50.0       # sigmoid rounds to 1
    l[7, 1::2] = 60.0
    l[8] = -200.0     # and to 0 in fp32
    b = None if bias is None else np.full(E, bias, dtype=np.float32)
    for by in ("max", "top2"):
        _check(l, k, b, scoring=scoring, groups=groups, kept=kept, by=by)


def test_shut_off_and_not_finite():
    rng = np.random.default_rng(8)
    l = _logits(rng, 12, 32)
    bias = np.zeros(32, dtype=np.float32)
    bias[4:30] = -np.inf
    for scoring in ("softmax", "sigmoid"):
        _check(l, 8, bias, scoring=scoring)                        # six open, two more in order of their index
        _check(l, 8, bias, scoring=scoring, groups=4, kept=1, by="top2")
        m = l.copy()
        m[0, 5] = np.inf
        _check(m, 4, None, scoring=scoring)
        _check(m, 4, None, scoring=scoring, renorm=False)
        m[3, 7] = np.nan
        _check(m, 4, None, status=-6, scoring=scoring)
        worse = np.zeros(32, dtype=np.float32)
        worse[9], worse[10] = np.nan, np.inf
        _check(l, 4, worse, status=-6, scoring=scoring)


def test_small_scores_keep_their_weights():
    """Weights over the chosen ones where every score is far below fp32's range."""
    l = np.array([[-150.0, -151.0, -149.5, -400.0, -150.5, -152.0, -160.0, -170.0]], dtype=np.float32)
    for scoring in ("softmax", "sigmoid"):
        _check(l, 3, None, scoring=scoring)
        _check(l, 8, None, scoring=scoring)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (37, 8, 8), (130, 160, 6), (70, 384, 8), (33, 512, 5)])
def test_gradient(scoring, renorm, T, E, k):
    rng = np.random.default_rng(T)
    l = _logits(rng, T, E, masked=T > 1)
    D, sel, idx, _, ws = _run(l, k, scoring=scoring, renorm=renorm, scale=2.5)
    dw, aux = rng.normal(size=(T, k)).astype(np.float32), rng.normal(size=(T, E)).astype(np.float32)
    dev = [torch.from_numpy(a).cuda() for a in (l, idx, dw, aux)]
    ref = _block.select_grad(l, idx, dw.astype(np.float64), scoring, renorm, 2.5)
    s = _block.scores(l, scoring)
    size = 2.5 * np.abs(dw).sum(1, keepdims=True) * np.where(np.isin(np.arange(E), idx), 1.0, s)
    got = f64(mok.select_experts_backward(D, sel, *dev[:3], ws))
    assert (np.abs(got - ref) <= G_REL * size + 1e-37).all()
    assert (got[~(l > -1e30)] == 0).all()
    got = f64(mok.select_experts_backward(D, sel, *dev[:3], ws, dlogits_aux=dev[3]))
    assert (np.abs(got - ref - aux) <= G_REL * size + 2.0 ** -23 * (np.abs(aux) + np.abs(ref))).all()
    assert mok.read_status(ws) == 0


def test_gradient_with_indices_out_of_range_and_twice():
    rng = np.random.default_rng(2)
    l = _logits(rng, 6, 16)
    D, sel, idx, _, ws = _run(l, 4, scoring="sigmoid")
    idx[1, 2], idx[2, 0], idx[3] = -1, 16, 7
    idx[4, 3] = idx[4, 0]
    dw = rng.normal(size=(6, 4)).astype(np.float32)
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            sel = mok.Selection(scoring=scoring, renormalise=renorm)
            mok.clear_status(ws)
            got = f64(mok.select_experts_backward(D, sel, *(torch.from_numpy(a).cuda() for a in (l, idx, dw)), ws))
            ref = _block.select_grad(l, idx, dw.astype(np.float64), scoring, renorm)
            assert np.abs(got - ref).max() <= G_REL * np.abs(dw).sum(1).max()
            assert mok.read_status(ws) == -6


def test_empty_batch_captured_graph_and_other_stream():
    ensure_lib()
    D0, sel = mok.dims(0, 128, 8, 2, 128, 0, 0), mok.Selection("sigmoid", scale=2.0)
    none = torch.empty((0, 8), device="cuda")
    idx, w = mok.select_experts(D0, sel, none, _ws())
    assert idx.shape == (0, 2) and mok.select_experts_backward(D0, sel, none, idx, w, _ws()).shape == (0, 8)
    rng = np.random.default_rng(9)
    D, l = mok.dims(64, 128, 64, 6, 128, 0, 0), torch.empty((64, 64), device="cuda")
    b, dw, ws = torch.zeros(64, device="cuda"), torch.ones((64, 6), device="cuda"), _ws()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            idx, w = mok.select_experts(D, sel, l, ws, bias=b)
            dl = mok.select_experts_backward(D, sel, l, idx, dw, ws)
        for _ in range(3):
            a = _logits(rng, 64, 64)
            l.copy_(torch.from_numpy(a))
            graph.replay()
            s.synchronize()
            ref, wref = _block.select(a, 6, "sigmoid", bias=np.zeros(64, np.float32), scale=2.0)
            assert np.array_equal(idx.cpu().numpy(), ref) and np.abs(f64(w) - wref).max() <= 2 * W_REL
            assert np.abs(f64(dl) - _block.select_grad(a, ref, f64(dw), "sigmoid", True, 2.0)).max() <= G_REL * 12


LAYER = LayerShape("select", 190, 256, 16, 4, 256, 256, 1, 0.0, "none", "bf16", True, 61)


@pytest.mark.parametrize("scoring,renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", False)])
@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_layer_with_a_selection(scoring, renorm, dtype):
    """The whole layer, trained through its weights: against autograd in 64 bits (bf16), and the
    logits' gradient against the operator's own for both types."""
    ensure_lib()
    D = dims_of(LAYER, dtype=mok.MOK_MXFP8 if dtype == "mxfp8" else mok.MOK_BF16)
    L = make_layer(LAYER, "cpu", with_dy=True)
    W = to_dev(L)
    x, dY = W.pop("x"), W.pop("dY")
    W["balance_bias"] = torch.linspace(-0.02, 0.02, 16, device="cuda")
    if dtype == "mxfp8":
        W["prepared"], W["prepared_bwd"] = mok.prepare_weights(D, W), mok.prepare_weights_bwd(D, W)
    sel = mok.Selection(scoring, n_groups=4, topk_groups=2, group_score="top2", renormalise=renorm, scale=2.5)
    layer = mok.MoELayer(D, W, selection=sel)
    y = layer.forward(x, training=True)
    aux = torch.full((190, 16), 1e-3, device="cuda")
    g, g_aux = layer.backward(x, dY), layer.backward(x, dY, dlogits_aux=aux)
    assert mok.read_status(layer.ws) == 0 and mok.read_status(layer._ws_bwd) == 0
    assert torch.equal(g_aux["dlogits"], g["dlogits"] + aux)
    idx = layer.routing["topk_idx"].long().cpu()
    logits = layer.logits.cpu().numpy()
    ref, wref = _block.select(logits, 4, scoring, bias=f64(W["balance_bias"]).astype(np.float32), groups=4, kept=2,
                              by="top2", renorm=renorm, scale=2.5)
    assert np.array_equal(idx.numpy(), ref)
    assert np.abs(f64(layer.routing["topk_w"]) - wref).max() <= W_REL * wref.max()

    P = {k: L[k].double().requires_grad_() for k in ("x", "W_router", "W_gate", "W_up", "W_down", "Ws_gate", "Ws_up", "Ws_down")}
    l = P["x"] @ P["W_router"]
    s = torch.sigmoid(l) if scoring == "sigmoid" else torch.softmax(l, 1)
    w = s.gather(1, idx)
    w = 2.5 * (w / w.sum(1, keepdim=True) if renorm else w)

    def ffn(v, a, b, c):
        return (torch.nn.functional.silu(v @ a) * (v @ b)) @ c

    out = ffn(P["x"], P["Ws_gate"], P["Ws_up"], P["Ws_down"])
    for e in range(16):
        rows, slots = (idx == e).nonzero(as_tuple=True)
        out = out.index_add(0, rows, w[rows, slots, None] * ffn(P["x"][rows], P["W_gate"][e], P["W_up"][e], P["W_down"][e]))
    grads = dict(zip(["dl", "w", *P], torch.autograd.grad((out * L["dY"].double()).sum(), [l, w, *P.values()])))
    if dtype == "mxfp8":  # E4M3 steps in the experts: looser, the structure is what counts here
        assert_close("dlogits", f64(g["dlogits"]), f64(grads["dl"]), 0.2, 0.1)
        return
    assert_close("y", f64(y), f64(out))
    assert_close("dlogits", f64(g["dlogits"]), f64(grads["dl"]))
    assert_close("dX", f64(g["dX"]), f64(grads["x"]))
    for k in ("W_router", "W_gate", "W_down", "Ws_up"):
        assert_close(k, f64(g["d" + k]), f64(grads[k]))
    plain = _block.select_grad(logits, ref, f64(grads["w"]), scoring, renorm, 2.5)
    assert_close("dlogits from dw", plain, f64(grads["dl"]), 1e-3, 1e-3)


def test_layer_with_experts_shut_off_by_the_routers_bias():
    """Fewer open experts than k: weights 0 for the others and nothing to report."""
    ensure_lib()
    D = dims_of(LAYER)
    W = to_dev(make_layer(LAYER, "cpu"))
    x = W.pop("x")
    W["bias"] = torch.full((16,), -float("inf"), device="cuda")
    W["bias"][[3, 11]] = 0.5
    layer = mok.MoELayer(D, W, selection=mok.Selection("sigmoid", scale=2.0))
    y = layer.forward(x)
    assert mok.read_status(layer.ws) == 0 and torch.isfinite(y).all()
    idx, w = (layer.routing[k].cpu() for k in ("topk_idx", "topk_w"))
    assert (idx[:, 2:] == torch.tensor([0, 1])).all() and (w[:, 2:] == 0).all()
    assert (idx[:, :2].sort(1).values == torch.tensor([3, 11])).all() and np.abs(f64(w[:, :2].sum(1)) - 2.0).max() < 1e-5
    logits = mok.route(D, x, W["W_router"], W["bias"], layer.ws, want_topk=False)
    assert logits[:2] == (None, None) and torch.equal(logits[2], layer.logits)


def test_more_than_2_31_logits():
    ensure_lib()
    T, E, n = 5600000, 384, 7
    l = torch.zeros((T, E), device="cuda")
    l[-n:] = torch.randn((n, E), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    D, few, sel = mok.dims(T, 128, E, 8, 128, 0, 0), mok.dims(n, 128, E, 8, 128, 0, 0), mok.Selection("sigmoid", scale=2.0)
    ws, b = _ws(), torch.zeros(E, device="cuda")
    idx, w = mok.select_experts(D, sel, l, ws, bias=b)
    i, v = mok.select_experts(few, sel, l[-n:].clone(), ws, bias=b)
    assert torch.equal(idx[-n:], i) and torch.equal(w[-n:], v) and (idx[:1000].cpu() == torch.arange(8)).all()
    dw = torch.zeros((T, 8), device="cuda")
    dw[-n:] = 1.0
    dw[-n:, 0] = 3.0
    dl = mok.select_experts_backward(D, sel, l, idx, dw, ws)
    assert torch.equal(dl[-n:], mok.select_experts_backward(few, sel, l[-n:].clone(), i, dw[-n:].clone(), ws))
    assert not dl[:1000].any() and mok.read_status(ws) == 0
