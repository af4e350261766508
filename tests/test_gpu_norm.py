"""RMS norm with the residual's addition and MXFP8 output, and its gradients, against 64 bits.

Tolerances.  u = 2^-24.  A thread adds at most 32 squares, then come 5 shuffles and at most 32
warps, so sums carry less than 128 u relative to the sum of magnitudes; with the root, the division
and two products v is within 80 u of its value.  A bf16 output is the rounding of such a value, so it
lies between the roundings of the two ends of that interval.
"""

import subprocess
import sys

import numpy as np
import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests import _around as plain
from tests._helpers import ROOT, ensure_lib, f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rows(T, d, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn((T, d), generator=g) * scale * torch.exp(0.5 * torch.randn((T, 1), generator=g))
    v[:, ::max(1, d // 3)] *= 30.0
    return v.to(dtype)


def _weight(d, dtype, seed):
    return (1.0 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(seed))).to(dtype)


def _rounds_to(got, want, noise):
    """Every bf16 of ``got`` is the rounding of some value within ``noise`` of ``want``."""
    low, high = (f64(torch.from_numpy(want + sign * noise).to(torch.bfloat16)) for sign in (-1, 1))
    got = f64(got)
    return ((low <= got) & (got <= high)).all()


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


SHAPES = [(1, 8), (1, 7168), (3, 72), (5, 256), (130, 128), (33, 2056), (7, 7168), (64, 1000), (2, 8200), (3, 32768),
          (700, 384), (1, 264)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("res", ["none", "bf16", "f32"])
@pytest.mark.parametrize("wt", ["bf16", "f32"])
def test_forward(T, d, res, wt):
    ensure_lib()
    x, w = _rows(T, d, torch.bfloat16, 1), _weight(d, TYPES[wt], 2)
    r = None if res == "none" else _rows(T, d, TYPES[res], 3, 4.0)
    xc, wc, rc = _cuda(x, w, r)
    out = mok.rms_norm(xc, wc, EPS, residual=rc)
    v, h = plain.rms_norm(f64(x), f64(w), EPS, None if r is None else f64(r))
    assert _rounds_to(out["y"], v, 80 * U * np.abs(v))
    if r is None:
        assert "residual" not in out
    elif res == "f32":
        assert torch.equal(out["residual"].cpu(), x.float() + r)
    else:
        assert torch.equal(out["residual"].cpu(), (x.float() + r.float()).to(torch.bfloat16))


@pytest.mark.parametrize("T,d", [(1, 128), (1, 7168), (5, 256), (129, 384), (300, 2048), (2, 32768)])
@pytest.mark.parametrize("res", ["none", "f32"])
@pytest.mark.parametrize("want_y", [True, False])
def test_mxfp8_output(T, d, res, want_y):
    """Codes within half a code of v at the scale of its block's amax; both scale layouts agree."""
    ensure_lib()
    x, w = _rows(T, d, torch.bfloat16, 4), _weight(d, torch.float32, 5)
    x[0, :32] = 0                                          # a block of zeros
    r = None if res == "none" else _rows(T, d, torch.float32, 6)
    if r is not None:
        r[0, :32] = 0
    xc, wc, rc = _cuda(x, w, r)
    rows = mok.rms_norm(xc, wc, EPS, residual=rc, mx="rows", want_y=want_y)
    atoms = mok.rms_norm(xc, wc, EPS, residual=rc, mx="atoms", want_y=want_y)
    assert ("y" in rows) == want_y
    v, _ = plain.rms_norm(f64(x), f64(w), EPS, None if r is None else f64(r))
    s, amax = plain.mx_exponents(v)
    got = rows["scales"].cpu().numpy().astype(np.int64) - 127
    edge = np.abs(np.log2(np.maximum(amax, 1e-300) / 448.0) - np.round(np.log2(np.maximum(amax, 1e-300) / 448.0))) < 1e-4
    assert ((got == s) | (edge & (np.abs(got - s) <= 1))).all()
    assert got[0, 0] == -127 and (rows["codes"][0, :32] == 0).all()
    scale = np.repeat(2.0 ** got, 32, axis=1)
    q = plain.e4m3(rows["codes"].cpu().numpy()) * scale
    assert (np.abs(q - v) <= (2.0 ** -4 + 80 * U) * np.abs(v) + 2.0 ** -10 * scale * 1.001).all()
    assert torch.equal(rows["codes"], atoms["codes"])
    tiles = atoms["scales"].cpu().numpy().reshape(-1, d // 128, 32, 4, 4)   # tile, K block, r0, r1, byte
    flat = tiles.transpose(0, 3, 2, 1, 4).reshape(-1, d // 32)              # row = 32 r1 + r0
    assert (flat[:T] == rows["scales"].cpu().numpy()).all() and (flat[T:] == 0).all()
    if want_y:
        assert _rounds_to(rows["y"], v, 80 * U * np.abs(v))


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("res", ["none", "bf16", "f32"])
@pytest.mark.parametrize("wt", ["bf16", "f32"])
def test_backward(T, d, res, wt):
    ensure_lib()
    kind = torch.float32 if res == "f32" else torch.bfloat16
    s, dy, w = _rows(T, d, kind, 7), _rows(T, d, torch.bfloat16, 8, 0.1), _weight(d, TYPES[wt], 9)
    dres = None if res == "none" else _rows(T, d, kind, 10, 0.1)
    sc, dyc, wc, dc = _cuda(s, dy, w, dres)
    out = mok.rms_norm_backward(dyc, sc, wc, EPS, dres=dc)
    S, DY, W = f64(s), f64(dy), f64(w)
    ds, dw = plain.rms_norm_grad(DY, S, W, EPS, None if dres is None else f64(dres))
    rho = 1.0 / np.sqrt((S * S).mean(1, keepdims=True) + EPS)
    size = rho * (np.abs(DY * W) + np.abs(S) * rho * (np.abs(DY * W * S) * rho).mean(1, keepdims=True))
    if dres is not None:
        size += np.abs(f64(dres))
    noise = 256 * U * size
    assert _rounds_to(out["dx"], ds, noise)
    if res == "f32":
        assert (np.abs(f64(out["dresidual"]) - ds) <= noise + 1e-30).all()
    else:
        assert "dresidual" not in out
    # rows are summed over at most T terms in a thread, then over the partial rows
    assert (np.abs(f64(out["dweight"]) - dw) <= (80 + T + 700) * U * (np.abs(DY * S) * rho).sum(0) + 1e-30).all()
    again = mok.rms_norm_backward(dyc, sc, wc, EPS, dres=dc)
    assert all(torch.equal(out[k], again[k]) for k in out)


def test_gradient_against_differences():
    """<gradient, direction> against a central difference of the 64-bit form."""
    ensure_lib()
    T, d = 37, 264
    s, dy, w = _rows(T, d, torch.float32, 11), _rows(T, d, torch.bfloat16, 12), _weight(d, torch.float32, 13)
    dres = _rows(T, d, torch.float32, 14)
    out = mok.rms_norm_backward(*_cuda(dy, s, w), EPS, dres=dres.cuda())
    rng = np.random.default_rng(0)
    u, uw = rng.standard_normal((T, d)) * np.abs(f64(s)).mean(1, keepdims=True), rng.standard_normal(d)

    def f(t):
        y, h = plain.rms_norm(f64(s) + t * u, f64(w) + t * uw, EPS)
        return (f64(dy) * y).sum() + (f64(dres) * h).sum()

    step = 1e-5
    want = (f(step) - f(-step)) / (2 * step)
    got = (f64(out["dresidual"]) * u).sum() + (f64(out["dweight"]) * uw).sum()
    size = np.abs(f64(out["dresidual"]) * u).sum() + np.abs(f64(out["dweight"]) * uw).sum()
    assert abs(got - want) <= 1e-5 * size      # 256 u of arithmetic and the difference's own 1e-8


def test_in_place_and_side_stream():
    ensure_lib()
    T, d = 65, 1024
    x, r, w = _cuda(_rows(T, d, torch.bfloat16, 15), _rows(T, d, torch.float32, 16), _weight(d, torch.float32, 17))
    want = mok.rms_norm(x, w, EPS, residual=r)
    x2, r2 = x.clone(), r.clone()
    L = mok.lib()
    assert L.mok_rms_norm(T, d, EPS, x2.data_ptr(), r2.data_ptr(), 1, w.data_ptr(), 1, x2.data_ptr(), r2.data_ptr(),
                          None, None, 0, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(x2, want["y"]) and torch.equal(r2, want["residual"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mok.rms_norm(x, w, EPS, residual=r)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got["y"], want["y"])


@pytest.mark.parametrize("T,d", [(700, 1024), (400, 7168), (330, 24576)])
@pytest.mark.parametrize("over", ["dres", "s"])
def test_backward_in_place(T, d, over):
    """dx over dy, dresidual over dres or over s, with and without rows in shared memory."""
    ensure_lib()
    s, dy, w, dres = _cuda(_rows(T, d, torch.float32, 30), _rows(T, d, torch.bfloat16, 31), _weight(d, torch.float32, 32),
                           _rows(T, d, torch.float32, 33))
    want = mok.rms_norm_backward(dy, s, w, EPS, dres=dres)
    ws = torch.zeros(mok.rms_norm_workspace_size(T, d), dtype=torch.uint8, device="cuda")
    dweight = torch.empty(d, device="cuda")
    target = dres if over == "dres" else s
    assert mok.lib().mok_rms_norm_backward(T, d, EPS, dy.data_ptr(), s.data_ptr(), 1, w.data_ptr(), 1, dres.data_ptr(),
                                           dy.data_ptr(), target.data_ptr(), dweight.data_ptr(), ws.data_ptr(),
                                           ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(dy, want["dx"]) and torch.equal(target, want["dresidual"]) and torch.equal(dweight, want["dweight"])


def test_zero_rows_and_non_finite_rows():
    """A zero row gives zeros; a row with inf or NaN does not touch the others."""
    ensure_lib()
    x, w = _rows(6, 256, torch.bfloat16, 18), _weight(256, torch.float32, 19)
    clean = mok.rms_norm(*_cuda(x, w), EPS, mx="rows")
    x[1], x[3, 5], x[4, 7] = 0, float("nan"), float("inf")
    out = mok.rms_norm(*_cuda(x, w), EPS, mx="rows")
    assert (out["y"][1] == 0).all() and (out["codes"][1] == 0).all() and (out["scales"][1] == 0).all()
    assert out["y"][3].isnan().all() and ((out["codes"][3] & 127) == 127).all()
    for t in (0, 2, 5):
        assert torch.equal(out["y"][t], clean["y"][t]) and torch.equal(out["codes"][t], clean["codes"][t])
    empty = mok.rms_norm(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), w.cuda(), EPS, mx="atoms")
    assert empty["y"].shape == (0, 256)
    g = mok.rms_norm_backward(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"),
                              torch.empty((0, 256), dtype=torch.float32, device="cuda"), w.cuda(), EPS)
    assert (g["dweight"] == 0).all()


WIDTHS = """
import torch
import mixture_experts_layer_14_gb300 as mok
T = 330
for d in [*range(8, 600, 72), *range(1024, 5400, 152), *range(5440, 17000, 992), 24000, 32760]:
    x = torch.randn(T, d, device="cuda").bfloat16()
    w = torch.ones(d, device="cuda")
    for kind in (None, torch.bfloat16, torch.float32):
        r = None if kind is None else torch.randn(T, d, device="cuda").to(kind)
        h = x.float() if r is None else x.float() + r.float()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6)
        out = mok.rms_norm(x, w, 1e-6, residual=r)
        assert (out["y"].float() - y).abs().max() <= 2 ** -7 * y.abs().max(), (d, kind)
        s = out.get("residual", x)
        g = mok.rms_norm_backward(x, s, w, 1e-6, dres=None if r is None else s)
        assert g["dx"].isfinite().all() and g["dweight"].isfinite().all(), (d, kind)
torch.cuda.synchronize()
"""


def test_every_width_in_a_fresh_process():
    """Shared-memory sizes on both sides of what a launch gets unasked: each kernel's first launch in
    the process is with the smaller ones."""
    ensure_lib()
    r = subprocess.run([sys.executable, "-c", WIDTHS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_offsets_beyond_32_bits():
    """T d > 2^31: the last rows are right (17 GB on the device)."""
    ensure_lib()
    T, d = 65600, 32768
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    x[:-3], tail = 1.0, _rows(3, d, torch.bfloat16, 20)
    x[-3:] = tail.cuda()
    w = _weight(d, torch.float32, 21)
    out = mok.rms_norm(x, w.cuda(), EPS, mx="atoms")
    v, _ = plain.rms_norm(f64(tail), f64(w), EPS)
    assert _rounds_to(out["y"][-3:], v, 80 * U * np.abs(v))
    small = mok.rms_norm(tail.cuda(), w.cuda(), EPS, mx="rows")
    assert torch.equal(out["codes"][-3:], small["codes"])
    del out
    g = mok.rms_norm_backward(x, x, w.cuda(), EPS)
    want = mok.rms_norm_backward(tail.cuda(), tail.cuda(), w.cuda(), EPS)
    assert torch.equal(g["dx"][-3:], want["dx"])
