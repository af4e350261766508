"""The norm after a branch, its gate, the scaled residual and the next norm, and their gradients,
against the plain 64-bit forms."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests import _around, _block
from tests._helpers import ensure_lib, f64

pytestmark = pytest.mark.gpu

A = 0.75
# Roundings to bf16 are half a step, 2^-8 of the value; fp32 arithmetic on top: each sum of d terms is
# taken in at most d / 1024 + 40 additions of 2^-24 (lanes, shuffles, warps), which enters the root by
# half, and about ten products: 2^-18 up to d = 32768 with cancellation against the row's size.
BF16 = 2.0 ** -8
F32 = 2.0 ** -18


def _close(got, ref, rel, size):
    got = f64(got)
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= rel * np.abs(ref) + F32 * size).all(), np.abs(got - ref).max()


def _make(T, d, res, w, gate, seed=0):
    g = torch.Generator().manual_seed(seed)
    rt, wt = (torch.float32 if k == "f32" else torch.bfloat16 for k in (res, w))
    v = dict(x=torch.randn((T, d), generator=g).bfloat16(), post=(1 + 0.1 * torch.randn(d, generator=g)).to(wt),
             weight=(1 + 0.1 * torch.randn(d, generator=g)).to(wt), gate=None, token_gate=None)
    r = torch.randn((T, d), generator=g) * torch.exp(0.5 * torch.randn((T, 1), generator=g))
    r[:, ::max(1, d // 5)] *= 20.0
    v["r"] = r.to(rt)
    if gate in ("channel", "both"):
        v["gate"] = (0.5 + 0.1 * torch.randn(d, generator=g)).to(wt)
    if gate in ("token", "both"):
        v["token_gate"] = torch.rand(T, generator=g)
        v["token_gate"][0] = 0.0
    return v


def _dev(v):
    return {k: t.cuda() if t is not None else None for k, t in v.items()}


def _np(v):
    return {k: f64(t) for k, t in v.items() if t is not None}


def _packed(t):
    """Codes and scales of a tensor by the 64-bit rule, and the values that they hold."""
    a = f64(t)
    s, _ = _around.mx_exponents(a)
    q = torch.from_numpy(a / np.repeat(2.0 ** s, 32, axis=-1)).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    return (q.view(torch.uint8).cuda(), torch.from_numpy((s + 127).astype(np.uint8)).cuda(),
            q.double().numpy() * np.repeat(2.0 ** s, 32, axis=-1))


CASES = [(1, 8, "bf16", "bf16", "none"), (1, 7168, "bf16", "bf16", "none"), (3, 256, "f32", "bf16", "both"),
         (9, 264, "bf16", "f32", "channel"), (700, 64, "bf16", "bf16", "token"), (517, 1544, "f32", "f32", "both"),
         (400, 4096, "bf16", "bf16", "channel"), (330, 7168, "f32", "bf16", "token"), (7, 8200, "bf16", "f32", "both"),
         (310, 16384, "bf16", "bf16", "none"), (5, 16392, "f32", "f32", "both"), (157, 32768, "bf16", "bf16", "token"),
         (2500, 128, "f32", "bf16", "none"), (311, 8192, "bf16", "bf16", "channel"), (5, 8448, "f32", "f32", "both"),
         # many rows per block, several times around the ring
         (1300, 4096, "f32", "bf16", "both"), (2500, 2056, "bf16", "f32", "channel"), (9001, 512, "bf16", "bf16", "token"),
         (20011, 128, "f32", "bf16", "none"), (1100, 7168, "f32", "bf16", "none"), (1500, 8192, "bf16", "bf16", "both"),
         (1300, 5120, "bf16", "f32", "both"), (1301, 4360, "f32", "bf16", "channel")]


@pytest.mark.parametrize("T,d,res,w,gate", CASES)
@pytest.mark.parametrize("next_norm", [True, False])
def test_forward(T, d, res, w, gate, next_norm):
    ensure_lib()
    v = _make(T, d, res, w, gate)
    if not next_norm:
        v["weight"] = None
    n, t = _np(v), _dev(v)
    out = mok.sandwich_norm(t["x"], t["r"], t["post"], weight=t["weight"], gate=t["gate"], token_gate=t["token_gate"],
                            res_scale=A)
    h, y = _block.sandwich(**n, a=A)
    size = np.abs(A * n["r"]) + np.abs(h - A * n["r"])
    _close(out["residual"], h, BF16 if res == "bf16" else 0.0, size)
    assert ("y" in out) == next_norm
    if next_norm:
        _close(out["y"], y, BF16, np.abs(y) + size * np.abs(n["weight"]) / np.sqrt((h * h).mean(1, keepdims=True)))


@pytest.mark.parametrize("T,d,res,gate,mx,want_y", [
    (1, 128, "bf16", "none", "rows", True), (130, 256, "f32", "both", "atoms", True), (33, 384, "bf16", "channel", "atoms", False),
    (301, 7168, "bf16", "token", "rows", False), (1301, 5120, "f32", "both", "rows", True), (3, 16512, "f32", "none", "atoms", True)])
def test_codes_and_checkpoint(T, d, res, gate, mx, want_y):
    """The MXFP8 output and the 8-bit forms of x and h: x's exactly; the others within half a step of
    their code (2^-4 of the value, 2^-10 of the scale below the smallest normal), and fp32 roundings
    that may choose the neighbour of a value halfway."""
    ensure_lib()
    v = _make(T, d, res, "bf16", gate, 1)
    v["r"][0] = 0
    v["x"][0, :64] = 0
    n, t = _np(v), _dev(v)
    args = dict(weight=t["weight"], gate=t["gate"], token_gate=t["token_gate"], res_scale=A)
    out = mok.sandwich_norm(t["x"], t["r"], t["post"], **args, mx=mx, want_y=want_y, save="mxfp8")
    plain = mok.sandwich_norm(t["x"], t["r"], t["post"], **args)
    assert torch.equal(out["residual"], plain["residual"]) and ("y" in out) == want_y
    assert not want_y or torch.equal(out["y"], plain["y"])
    codes, scales, _ = _packed(v["x"])
    assert torch.equal(out["x_codes"], codes) and torch.equal(out["x_scales"], scales)
    h, y = _block.sandwich(**n, a=A)
    size = np.abs(A * n["r"]) + np.abs(h - A * n["r"])
    rows = out["scales"].cpu().numpy() if mx == "rows" else None
    if mx == "atoms":
        flat, tile = out["scales"].cpu().numpy().reshape(-1, d // 128, 32, 4, 4), np.arange((T + 127) // 128 * 128)
        rows = flat[tile // 128, :, tile % 32, tile % 128 // 32].reshape(len(tile), d // 32)
        assert (rows[T:] == 0).all()
        rows = rows[:T]
    for name, c, s, ref, slack in (("y", out["codes"], rows, y, np.abs(n["weight"]) / np.sqrt((h * h).mean(1, keepdims=True) + 1e-6)),
                                   ("h", out["h_codes"], out["h_scales"].cpu().numpy(), h, 1.0)):
        scale = np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, axis=1)
        got = _around.e4m3(c.cpu().numpy()) * scale
        assert (np.abs(got - ref) <= np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * scale) + 2 * F32 * size * slack).all(), name
        want, amax = _around.mx_exponents(ref)
        clear = np.abs(amax / 448.0 / 2.0 ** np.round(np.log2(np.maximum(amax, 1e-300) / 448.0)) - 1.0) > 2.0 ** -14
        assert (s.astype(np.int64) - 127 == want)[clear | (amax == 0)].all(), name


def test_checkpoint_without_a_next_norm():
    ensure_lib()
    t = _dev(_make(70, 384, "bf16", "f32", "both", 4))
    args = dict(gate=t["gate"], token_gate=t["token_gate"], res_scale=A)
    full = mok.sandwich_norm(t["x"], t["r"], t["post"], weight=t["weight"], save="mxfp8", **args)
    last = mok.sandwich_norm(t["x"], t["r"], t["post"], save="mxfp8", **args)
    assert set(last) == set(full) - {"y"} and all(torch.equal(last[k], full[k]) for k in last)


@pytest.mark.parametrize("T,d,res,w,gate", CASES)
@pytest.mark.parametrize("next_norm,dh,packed", [(True, True, False), (True, False, False), (False, True, False),
                                                 (True, True, True), (False, True, True)])
def test_backward(T, d, res, w, gate, next_norm, dh, packed):
    if packed and d % 128:
        pytest.skip("8-bit forms want d % 128 == 0")
    ensure_lib()
    v = _make(T, d, res, w, gate, 2)
    g = torch.Generator().manual_seed(3)
    if not next_norm:
        v["weight"] = None
    rt = v["r"].dtype
    dy = torch.randn((T, d), generator=g).bfloat16() * 0.01 if next_norm else None
    dres = (torch.randn((T, d), generator=g) * 0.01).to(rt) if dh else None
    h = v.pop("r")
    n, t = _np(v), _dev(v)
    n["h"], dev_x, dev_h = f64(h), t["x"], h.cuda()
    if packed:
        c, s, n["x"] = _packed(v["x"])
        dev_x = (c, s)
        c, s, n["h"] = _packed(h)
        dev_h = (c, s)
    out = mok.sandwich_norm_backward(
        dev_x, dev_h if next_norm else None, t["post"], dy=None if dy is None else dy.cuda(),
        dres=None if dres is None else dres.cuda(), weight=t["weight"], gate=t["gate"], token_gate=t["token_gate"],
        res_scale=A, residual_dtype=rt)
    rest = {k: n[k] for k in ("weight", "gate", "token_gate") if k in n}
    f = lambda a: None if a is None else f64(a)  # noqa: E731
    ref = _block.sandwich_grad(n["x"], n["h"], n["post"], f(dy), f(dres), a=A, **rest)
    assert set(out) == set(ref)
    # sizes of the terms that are subtracted: per row for dx and ds, summed over rows for the weights
    ds = np.abs(ref["dresidual"]) / A + (0.0 if dres is None else np.abs(f64(dres)))
    rowmax = np.abs(ref["dresidual"]).max(1, keepdims=True) / A + ds.max(1, keepdims=True)
    rho = 1.0 / np.sqrt((n["x"] ** 2).mean(1, keepdims=True) + 1e-6)
    W = np.abs(n["post"] * n.get("gate", 1.0)).max()
    tg = n["token_gate"][:, None] if "token_gate" in n else 1.0
    xhat = np.abs(n["x"]) * rho
    _close(out["dresidual"], ref["dresidual"], BF16 if res == "bf16" else 0.0, 4 * rowmax)
    _close(out["dx"], ref["dx"], BF16, 4 * rowmax * W * rho * tg * (1 + xhat))
    total = (np.abs(tg) * 4 * rowmax * (1 + xhat)).sum(0)
    _close(out["dpost_weight"], ref["dpost_weight"], 0.0, total)
    if gate in ("channel", "both"):
        _close(out["dgate"], ref["dgate"], 0.0, total * W * 2)
    if gate in ("token", "both"):
        _close(out["dtoken_gate"], ref["dtoken_gate"], 0.0, (4 * rowmax * W * (1 + xhat)).sum(1))
    if next_norm:
        hh = np.abs(n["h"]) / np.sqrt((n["h"] ** 2).mean(1, keepdims=True) + 1e-6)
        _close(out["dweight"], ref["dweight"], 0.0, (np.abs(f64(dy)) * hh).sum(0) * 2)


def test_in_place_rerun_graph_and_empty():
    """residual_out may be residual and y may be x; dx may be dy and dresidual dres; the same
    bits in a captured graph with its own workspace; no rows at all."""
    L = ensure_lib()
    import ctypes
    T, d = 321, 1024
    v = _dev(_make(T, d, "f32", "bf16", "both", 5))
    out = mok.sandwich_norm(v["x"], v["r"], v["post"], weight=v["weight"], gate=v["gate"], token_gate=v["token_gate"])
    a = mok._sandwich((T, d), v["x"].device, 1, v["post"], v["weight"], v["gate"], v["token_gate"], 1.0, 1e-6)
    x, r = v["x"].clone(), v["r"].clone()
    mok._check(L.mok_sandwich_norm(ctypes.byref(a), T, d, x.data_ptr(), r.data_ptr(), r.data_ptr(), x.data_ptr(), None,
                                   None, 0, None, None, None, None, mok._stream()))
    assert torch.equal(x, out["y"]) and torch.equal(r, out["residual"])
    dy, dres = torch.randn_like(v["x"]), torch.randn_like(v["r"])
    args = dict(dy=dy, dres=dres, weight=v["weight"], gate=v["gate"], token_gate=v["token_gate"])
    want = mok.sandwich_norm_backward(v["x"], out["residual"], v["post"], **args)
    ws = torch.zeros(mok.sandwich_norm_workspace_size(T, d), dtype=torch.uint8, device="cuda")
    dx, dr = dy.clone(), dres.clone()
    w = [torch.empty(d, device="cuda") for _ in range(3)] + [torch.empty(T, device="cuda")]
    mok._check(L.mok_sandwich_norm_backward(
        ctypes.byref(a), T, d, dx.data_ptr(), dr.data_ptr(), v["x"].data_ptr(), None, out["residual"].data_ptr(), None,
        dx.data_ptr(), dr.data_ptr(), w[0].data_ptr(), w[1].data_ptr(), w[3].data_ptr(), w[2].data_ptr(), ws.data_ptr(),
        ws.numel(), mok._stream()))
    for got, k in ((dx, "dx"), (dr, "dresidual"), (w[0], "dpost_weight"), (w[1], "dgate"), (w[2], "dweight"), (w[3], "dtoken_gate")):
        assert torch.equal(got, want[k]), k
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            y = mok.sandwich_norm(v["x"], v["r"], v["post"], weight=v["weight"], gate=v["gate"],
                                  token_gate=v["token_gate"])
            g = mok.sandwich_norm_backward(v["x"], y["residual"], v["post"], **args, ws=ws)
        for _ in range(2):
            graph.replay()
        s.synchronize()
    assert torch.equal(y["y"], out["y"]) and all(torch.equal(g[k], want[k]) for k in want)
    none = {k: (t[:0] if k in ("x", "r", "token_gate") else t) for k, t in v.items()}
    y = mok.sandwich_norm(none["x"], none["r"], v["post"], weight=v["weight"], gate=v["gate"],
                          token_gate=none["token_gate"])
    g = mok.sandwich_norm_backward(none["x"], y["residual"], v["post"], dy=none["x"], weight=v["weight"],
                                   gate=v["gate"], token_gate=none["token_gate"])
    assert y["y"].shape == (0, d) and all((g[k] == 0).all() and g[k].shape == (d,) for k in ("dpost_weight", "dgate", "dweight"))


def test_rows_that_are_not_finite_stay_their_own():
    """A row with NaN or infinities spoils nothing but itself (and the weights' gradients)."""
    ensure_lib()
    v = _dev(_make(40, 512, "bf16", "bf16", "none", 6))
    clean = mok.sandwich_norm(v["x"], v["r"], v["post"], weight=v["weight"], save="mxfp8")
    x, r = v["x"].clone(), v["r"].clone()
    x[3, 5], r[17, 100] = float("nan"), float("inf")
    out = mok.sandwich_norm(x, r, v["post"], weight=v["weight"], save="mxfp8")
    ok = torch.ones(40, dtype=torch.bool, device="cuda")
    ok[3] = ok[17] = False
    assert all(torch.equal(out[k][ok], clean[k][ok]) for k in clean)
    assert out["y"][3].isnan().all() and out["y"][17].isnan().any()
    dy = torch.randn_like(x)
    a = mok.sandwich_norm_backward(v["x"], clean["residual"], v["post"], dy=dy, weight=v["weight"])
    b = mok.sandwich_norm_backward(x, out["residual"], v["post"], dy=dy, weight=v["weight"])
    assert torch.equal(a["dx"][ok], b["dx"][ok]) and torch.equal(a["dresidual"][ok], b["dresidual"][ok])


def test_more_than_2_31_elements():
    """The last rows of a tensor whose offsets pass 32 bits, against the same rows by themselves."""
    ensure_lib()
    T, d, n = 262400, 8192, 5
    post, w = torch.linspace(0.5, 1.5, d, device="cuda"), torch.linspace(1.5, 0.5, d, device="cuda")
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    r = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(9)
    for t in (x, r):
        t[-n:] = torch.randn((n, d), generator=g, device="cuda").bfloat16()
    out = mok.sandwich_norm(x, r, post, weight=w, save="mxfp8")
    few = mok.sandwich_norm(x[-n:].clone(), r[-n:].clone(), post, weight=w, save="mxfp8")
    assert all(torch.equal(out[k][-n:], few[k]) and not out[k][:1].float().any() for k in ("residual", "y", "x_codes", "h_codes"))
    assert all(torch.equal(out[k][-n:], few[k]) for k in ("x_scales", "h_scales"))
    x8, h8 = ((out[k + "_codes"], out[k + "_scales"]) for k in ("x", "h"))
    few8 = [tuple(t[-n:].clone() for t in p) for p in (x8, h8)]
    del r, out["y"], out["residual"]
    dy = x  # the gradient of the last rows, zero elsewhere
    for a, b in ((x8, h8), few8):
        m = len(a[0])
        got = mok.sandwich_norm_backward(a, b, post, dy=dy[-m:] if m == T else dy[-n:].clone(), weight=w)
        if m == T:
            tail = {k: v[-n:].clone() if v.dim() == 2 else v for k, v in got.items()}
            assert not got["dx"][:1000].any()
            del got
    assert torch.equal(tail["dx"], got["dx"]) and torch.equal(tail["dresidual"], got["dresidual"])
    for k in ("dpost_weight", "dweight"):  # the same rows in another order of blocks
        size = got[k].abs().max()
        assert ((tail[k] - got[k]).abs() <= 2.0 ** -18 * size).all(), k
