"""Activations in 8 bits: packing and unpacking by the 64-bit rule, the layer's saved activations, and
blocks that train from them."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from mixture_experts_layer_14_gb300.synthetic import LayerShape, make_layer
from mixture_experts_layer_14_gb300.train_block import train
from tests import _around, _block
from tests._helpers import assert_close, dims_of, ensure_lib, f64, to_dev

pytestmark = pytest.mark.gpu

TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rule(a):
    """Codes, scale bytes and values by the 64-bit rule (torch rounds to the nearest code, ties to even)."""
    s, _ = _around.mx_exponents(a)
    wide = np.repeat(2.0 ** s, 32, axis=-1)
    q = torch.from_numpy(a / wide).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    return q.view(torch.uint8).numpy(), (s + 127).astype(np.uint8), q.double().numpy() * wide


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (257, 32), (1000, 2048), (33, 7168), (8200, 160)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_pack_and_unpack(rows, K, kind):
    ensure_lib()
    g = torch.Generator().manual_seed(rows)
    x = torch.randn((rows, K), generator=g) * torch.exp(3 * torch.randn((rows, 1), generator=g))
    x[0] = 0
    x[-1, :32] *= 2.0 ** -120
    x = x.to(TYPE[kind])
    codes, scales = mok.activation_pack(x.cuda())
    q, s, v = _rule(f64(x))
    assert np.array_equal(codes.cpu().numpy(), q) and np.array_equal(scales.cpu().numpy(), s)
    for out in ("bf16", "f32"):
        ref = torch.from_numpy(v).to(torch.float32).to(TYPE[out])
        assert torch.equal(mok.activation_unpack(codes, scales, TYPE[out]).cpu(), ref)
    buf = torch.full_like(x, 7.0).cuda()
    assert mok.activation_unpack(codes, scales, x.dtype, out=buf) is buf and torch.equal(buf.cpu(), torch.from_numpy(v).to(x.dtype))


def test_same_codes_as_the_layers_quantiser_and_atoms():
    ensure_lib()
    x = torch.randn((300, 256), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    codes, scales = mok.activation_pack(x.view(3, 100, 256))
    q, s = mok.mx_quantize_rows(x)
    assert torch.equal(codes.view(300, 256), q) and torch.equal(scales.view(300, 8), s)
    n = mok.rms_norm(x, torch.ones(256, device="cuda"), mx="atoms")
    r = mok.rms_norm(x, torch.ones(256, device="cuda"), mx="rows")
    for kind in TYPE.values():
        assert torch.equal(mok.activation_unpack(n["codes"], n["scales"], kind, layout="atoms"),
                           mok.activation_unpack(r["codes"], r["scales"], kind))


def test_every_code_and_scale_and_values_that_are_not_finite():
    ensure_lib()
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 8).cuda()
    v = _around.e4m3(np.arange(256))[None, :] * 2.0 ** (np.arange(256)[:, None] - 127.0)
    v[255] = np.nan
    for kind in TYPE.values():
        with np.errstate(over="ignore"):
            ref = torch.from_numpy(v.astype(np.float32)).to(kind)  # exact in fp32 but for overflow and 2^-136 ..
        got = mok.activation_unpack(codes, scales, kind).cpu()
        assert torch.equal(got.isnan(), ref.isnan()) and torch.equal(got.nan_to_num(1.0), ref.nan_to_num(1.0))
    x = torch.ones((2, 64))
    x[0, 3], x[1, 40] = float("nan"), float("inf")
    for kind in TYPE.values():
        c, s = mok.activation_pack(x.to(kind).cuda())
        back = mok.activation_unpack(c, s, kind).cpu()
        assert back[0, 3].isnan() and back[0].nan_to_num(1.0).eq(1).all() and back[1, :32].eq(1).all() and back[1, 40].isinf()


def test_empty_large_offsets_and_graph():
    """No rows; elements beyond 2^31; the same bits from a captured graph on another stream."""
    ensure_lib()
    c, s = mok.activation_pack(torch.empty((0, 64), device="cuda"))
    assert c.shape == (0, 64) and s.shape == (0, 2) and mok.activation_unpack(c, s).shape == (0, 64)
    x = torch.zeros(((1 << 20) + 3, 2048), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, 2048), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    c, s = mok.activation_pack(x)
    a, b = mok.activation_pack(x[-3:].clone())
    assert torch.equal(c[-3:], a) and torch.equal(s[-3:], b) and not c[:-3].any()
    assert torch.equal(mok.activation_unpack(c, s)[-3:], mok.activation_unpack(a, b))
    del x, c, s
    y, st = torch.randn((500, 96), device="cuda"), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            p = mok.activation_pack(y)
            z = mok.activation_unpack(*p, torch.float32)
        y.mul_(3.0)
        graph.replay()
        st.synchronize()
        want = mok.activation_pack(y)
    assert torch.equal(p[0], want[0]) and torch.equal(z, mok.activation_unpack(*want, torch.float32))


SHAPE = LayerShape("checkpoint", 200, 256, 16, 4, 256, 256, 1, 0.0, "normal0.1", "bf16", True, 71)
CODE = {"bf16": mok.MOK_BF16, "mxfp8": mok.MOK_MXFP8}


def _layer(dtype, n_shared=1, seed=71, **kw):
    shape = SHAPE.with_(dtype=dtype, n_shared=n_shared, F_shared=256 if n_shared else 0, cid=seed)
    D = dims_of(shape, dtype=CODE[dtype])
    W = to_dev(make_layer(shape, "cpu", with_dy=True))
    x, dY = W.pop("x"), W.pop("dY")
    if dtype == "mxfp8":
        W["prepared"], W["prepared_bwd"] = mok.prepare_weights(D, W), mok.prepare_weights_bwd(D, W)
    return D, W, x, dY


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
@pytest.mark.parametrize("n_shared", [1, 0])
def test_saved_activations(dtype, n_shared):
    """G and U come back as the values that their codes hold, x in expert order as it was; layers that
    share one buffer train as alone."""
    ensure_lib()
    D, W, x, dY = _layer(dtype, n_shared)
    plain = mok.MoELayer(D, W)
    y = plain.forward(x, training=True)
    before = plain.saved.clone()
    packed = mok.saved_pack(D, plain.saved)
    assert torch.equal(before, plain.saved)
    plain.saved.fill_(255)
    mok.saved_unpack(D, packed, x, plain.routing, plain.saved)
    kind, size = (torch.float32, 4) if dtype == "mxfp8" else (torch.bfloat16, 2)
    at = 0
    for n in [200 * 4 * 256] * 2 + [200 * 256] * (2 * n_shared):
        a, b = (t[at:at + size * n].view(kind) for t in (before, plain.saved))
        assert torch.equal(mok.activation_unpack(*mok.activation_pack(a), kind), b)
        at += (size * n + 1023) // 1024 * 1024
    if dtype == "bf16":
        assert torch.equal(before[at:at + 2 * 800 * 256], plain.saved[at:at + 2 * 800 * 256])
    want = plain.backward(x, dY)

    shared = torch.empty(mok.saved_size(D), dtype=torch.uint8, device="cuda")
    layers = [mok.MoELayer(D, W, checkpoint="mxfp8", saved=shared) for _ in range(2)]
    assert torch.equal(layers[0].forward(x, training=True), y)
    layers[1].forward(x.flip(0), training=True)
    layers[0].forward(3 * x)
    layers[1].backward(x.flip(0), dY)
    got = layers[0].backward(x, dY)
    assert all((want[k] is None and got[k] is None) or torch.equal(want[k], got[k]) for k in want)


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
@pytest.mark.parametrize("post,res", [(False, torch.bfloat16), (True, torch.float32), (True, torch.bfloat16), (False, None)])
def test_block_from_its_checkpoint(dtype, post, res):
    """A block that keeps 8 bits computes the gradients at the values that these hold: the same bits
    as the parts put together by hand; and not far from those of the block that keeps everything."""
    ensure_lib()
    D, W, x, dY = _layer(dtype)
    W["norm"] = torch.linspace(0.5, 1.5, 256, device="cuda")
    kw, tg = {}, None
    if post:
        W["post_norm"], W["post_gate"] = torch.linspace(1.5, 0.5, 256, device="cuda"), torch.linspace(0.1, 1.0, 256, device="cuda").bfloat16()
        kw, tg = dict(res_scale=0.8), torch.linspace(0.0, 1.0, 200, device="cuda")
    r = None if res is None else torch.randn(x.shape, generator=torch.Generator().manual_seed(1)).to(res).cuda()
    sel = mok.Selection("sigmoid", n_groups=4, topk_groups=2, group_score="top2", scale=2.5)
    full = mok.MoEBlock(D, W, alpha=0.1, z_coef=1e-2, selection=sel, **kw)
    b = mok.MoEBlock(D, W, alpha=0.1, z_coef=1e-2, selection=sel, checkpoint="mxfp8", **kw)
    y0, h0 = full.forward(x, r, training=True, token_gate=tg)
    y, h = b.forward(x, r, training=True, token_gate=tg)
    assert torch.equal(y, y0) and torch.equal(h, h0) and b.u is None
    dh = None if r is None else (r * 0.1)
    g0, g = full.backward(dY, dh), b.backward(dY, dh)
    assert set(g) == set(g0) and len(b.gradients(g)) == len(b.parameters()[0])
    for k in g:  # E4M3 rounds by up to 1/16, about 1/40 in the mean, in each of a few factors
        if g[k] is not None:
            ref = f64(g0[k])
            assert np.sqrt(((f64(g[k]) - ref) ** 2).sum() / (ref ** 2).sum()) < 0.15, k

    u8 = (lambda v: mok.activation_unpack(*mok.activation_pack(v), v.dtype))
    if post:
        n = mok.sandwich_norm(x, r, W["post_norm"], weight=W["norm"], gate=W["post_gate"], token_gate=tg, res_scale=0.8,
                              mx="rows", save="mxfp8")
    else:
        n = mok.rms_norm(x, W["norm"], residual=r, mx="rows")
    u = mok.activation_unpack(n["codes"], n["scales"])
    layer = mok.MoELayer(D, W, selection=sel, checkpoint="mxfp8")
    atoms = mok.rms_norm(x, W["norm"], residual=r, mx="atoms") if not post else mok.sandwich_norm(
        x, r, W["post_norm"], weight=W["norm"], gate=W["post_gate"], token_gate=tg, res_scale=0.8, mx="atoms")
    layer.forward(n["y"], training=True, x_mx=(atoms["codes"], atoms["scales"]) if dtype == "mxfp8" else None)
    want = layer.backward(u, dY, dlogits_aux=b.aux["dlogits"])
    assert torch.equal(want["dW_gate"], g["dW_gate"]) and torch.equal(want["dlogits"], g["dlogits"])
    if post:
        m = mok.sandwich_norm_backward((n["x_codes"], n["x_scales"]), (n["h_codes"], n["h_scales"]), W["post_norm"],
                                       dy=want["dX"], dres=dh, weight=W["norm"], gate=W["post_gate"], token_gate=tg,
                                       res_scale=0.8, residual_dtype=res)
        assert torch.equal(m["dpost_weight"], g["post_norm"]) and torch.equal(m["dgate"], g["post_gate"])
        assert torch.equal(m["dtoken_gate"], g["token_gate"]) and torch.equal(m["dresidual"], g["dresidual"])
    else:
        m = mok.rms_norm_backward(want["dX"], u8(h), W["norm"], dres=dh)
    assert torch.equal(m["dx"], g["dinput"]) and torch.equal(m["dweight"], g["norm"])


def test_block_with_norms_on_both_sides_against_autograd():
    """The whole bf16 block, sigmoid selection with groups, gates, residual scale and losses off, in
    64 bits."""
    ensure_lib()
    D, W, x, dY = _layer("bf16")
    W["norm"], W["post_norm"] = torch.linspace(0.5, 1.5, 256, device="cuda"), torch.linspace(1.5, 0.5, 256, device="cuda")
    W["post_gate"], tg = torch.linspace(0.2, 1.0, 256, device="cuda"), torch.linspace(0.1, 1.0, 200, device="cuda")
    r = torch.randn(x.shape, generator=torch.Generator().manual_seed(1)).cuda()
    dh = torch.randn(x.shape, generator=torch.Generator().manual_seed(2)).cuda() * 0.1
    sel = mok.Selection("sigmoid", scale=2.0)
    b = mok.MoEBlock(D, W, selection=sel, res_scale=0.8)
    y, h = b.forward(x, r, training=True, token_gate=tg)
    g = b.backward(dY, dh)
    idx = b.layer.routing["topk_idx"].long().cpu()
    names = ["W_router", "W_gate", "W_up", "W_down", "Ws_gate", "Ws_up", "Ws_down", "norm", "post_norm", "post_gate"]
    P = {k: W[k].double().cpu().requires_grad_() for k in names}
    P.update(x=x.double().cpu().requires_grad_(), r=r.double().cpu().requires_grad_(), tg=tg.double().cpu().requires_grad_())

    def unit(v):
        return v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt()

    def ffn(v, a, c, d):
        return (torch.nn.functional.silu(v @ a) * (v @ c)) @ d

    hh = 0.8 * P["r"] + P["tg"][:, None] * unit(P["x"]) * P["post_norm"] * P["post_gate"]
    u = unit(hh) * P["norm"]
    s = torch.sigmoid(u @ P["W_router"] + W["bias"].double().cpu()).gather(1, idx)
    w = 2.0 * s / s.sum(1, keepdim=True)
    out = ffn(u, P["Ws_gate"], P["Ws_up"], P["Ws_down"])
    for e in range(16):
        rows, slots = (idx == e).nonzero(as_tuple=True)
        out = out.index_add(0, rows, w[rows, slots, None] * ffn(u[rows], P["W_gate"][e], P["W_up"][e], P["W_down"][e]))
    grads = dict(zip(P, torch.autograd.grad((out * dY.double().cpu()).sum() + (hh * dh.double().cpu()).sum(), list(P.values()))))
    assert_close("y", f64(y), f64(out))
    assert_close("h", f64(h), f64(hh), 1e-5, 1e-5)
    ours = dict(x="dinput", r="dresidual", tg="token_gate", norm="norm", post_norm="post_norm", post_gate="post_gate")
    for k in P:
        assert_close(k, f64(g[ours.get(k, "d" + k)]), f64(grads[k]))


@pytest.mark.parametrize("kw", [dict(scoring="sigmoid", post_norm=True, checkpoint="mxfp8"), dict(scoring="softmax", dtype="mxfp8",
                                checkpoint="mxfp8"), dict(post_norm=True, states="mxfp8")])
def test_training_runs(kw):
    ensure_lib()
    assert np.isfinite(train(steps=3, **kw)).all()


def test_block_refusals():
    ensure_lib()
    D, W, x, dY = _layer("bf16")
    W["norm"] = torch.ones(256, device="cuda")
    small = torch.empty(8, dtype=torch.uint8, device="cuda")
    whole = torch.empty(mok.saved_size(D), dtype=torch.uint8, device="cuda")
    for bad in (dict(res_scale=0.5), dict(checkpoint="int8"), dict(saved=small, checkpoint="mxfp8"), dict(saved=whole)):
        with pytest.raises(ValueError):
            mok.MoEBlock(D, W, **bad)
    with pytest.raises(ValueError):
        mok.MoEBlock(D, W).forward(x, x, token_gate=torch.ones(200, device="cuda"))
    W["post_norm"] = torch.ones(256, device="cuda")
    with pytest.raises(ValueError):
        mok.MoEBlock(D, W).forward(x)
    with pytest.raises(mok.MokError):
        mok.MoELayer(D, W, checkpoint="mxfp8").backward(x, dY)
