"""RMS norm where a block takes several rows: the ring's places are filled again, the sums of the
next row are taken beside this row's outputs, dweight grows over a block's rows.

Tolerances.  u = 2^-24.  As for single rows: outputs are within 80 u (forward) or 256 u of the terms'
magnitudes (backward) before their rounding, which is monotone.  dweight: a block adds its T / blocks
rows, a thread of the second pass every 64th of the partial rows, then 2 shuffles and 16 warps, and
every term carries less than 80 u.
"""

import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests._helpers import ensure_lib

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rows(T, d, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn((T, d), generator=g, device="cuda") * scale
    v *= torch.exp(0.5 * torch.randn((T, 1), generator=g, device="cuda"))
    v[:, ::max(1, d // 3)] *= 30.0
    return v.to(dtype)


def _weight(d, dtype, seed):
    return (1.0 + 0.2 * torch.randn(d, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")).to(dtype)


def _rounds_to(got, want, noise):
    return (((want - noise).to(torch.bfloat16) <= got) & (got <= (want + noise).to(torch.bfloat16))).all()


def _check_backward(dy, s, w, dres):
    T, d = s.shape
    out = mok.rms_norm_backward(dy, s, w, EPS, dres=dres)
    S, DY, W = s.double(), dy.double(), w.double()
    rho = (S.square().mean(1, keepdim=True) + EPS) ** -0.5
    G = DY * W
    ds = rho * (G - S * rho * (G * S * rho).mean(1, keepdim=True))
    size = rho * (G.abs() + (S * rho).abs() * (G * S * rho).abs().mean(1, keepdim=True))
    if dres is not None:
        ds += dres
        size += dres.double().abs()
    noise = 256 * U * size
    assert _rounds_to(out["dx"], ds, noise), (T, d)
    if s.dtype == torch.float32:
        assert ((out["dresidual"].double() - ds).abs() <= noise + 1e-30).all(), (T, d)
    blocks = (mok.rms_norm_workspace_size(T, d) - 256) // (4 * d)
    terms = (T + blocks - 1) // blocks + blocks / 64 + 1 + 2 + 16 + 80
    xhat = S * rho
    assert ((out["dweight"].double() - (DY * xhat).sum(0)).abs() <= terms * U * (DY * xhat).abs().sum(0) + 1e-30).all(), (T, d)
    return T / blocks


# T: several times the blocks that a GPU with 152 SMs runs at this width, and a remainder; the
# last two widths have two vectors and four per thread
MANY = [(3013, 264, 2), (2711, 1000, 2), (1511, 2056, 3), (1000, 4096, 3), (701, 7168, 4), (503, 9000, 3), (503, 24576, 3)]


@pytest.mark.parametrize("T,d,turns", MANY)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("with_dres", [False, True])
def test_backward_several_rows_per_block(T, d, turns, kind, with_dres):
    ensure_lib()
    s, dy, w = _rows(T, d, TYPES[kind], 1), _rows(T, d, torch.bfloat16, 2, 0.1), _weight(d, TYPES[kind], 3)
    assert _check_backward(dy, s, w, _rows(T, d, TYPES[kind], 4, 0.1) if with_dres else None) > turns


@pytest.mark.parametrize("T,d,turns", MANY)
@pytest.mark.parametrize("res", ["none", "bf16", "f32"])
def test_forward_several_rows_per_block(T, d, turns, res):
    ensure_lib()
    x, w = _rows(T, d, torch.bfloat16, 5), _weight(d, torch.float32, 6)
    r = None if res == "none" else _rows(T, d, TYPES[res], 7, 4.0)
    out = mok.rms_norm(x, w, EPS, residual=r)
    h = x.double() if r is None else x.double() + r.double()
    v = h * (h.square().mean(1, keepdim=True) + EPS) ** -0.5 * w.double()
    assert _rounds_to(out["y"], v, 80 * U * v.abs())
    if r is not None:
        assert torch.equal(out["residual"], (x.float() + r.float()).to(r.dtype))


def test_gradients_of_every_width():
    """Two to three rows per block at the widths on both sides of each kernel's limits."""
    ensure_lib()
    T = 330
    for d in [*range(8, 600, 72), *range(1024, 5400, 152), *range(5440, 17000, 992), 24000, 32760]:
        w = _weight(d, torch.float32, d)
        dy = _rows(T, d, torch.bfloat16, d + 1, 0.1)
        for kind, with_dres in ((torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, True)):
            s = _rows(T, d, kind, d + 2)
            _check_backward(dy, s, w, _rows(T, d, kind, d + 3, 0.1) if with_dres else None)


@pytest.mark.parametrize("T,d", [(1, 256), (129, 384), (3013, 256), (701, 7168)])
def test_mxfp8_output_with_a_bf16_residual(T, d):
    """Codes and scales of the unrounded sum's norm, in rows and in atoms."""
    ensure_lib()
    x, r, w = _rows(T, d, torch.bfloat16, 8), _rows(T, d, torch.bfloat16, 9, 4.0), _weight(d, torch.bfloat16, 10)
    rows, atoms = (mok.rms_norm(x, w, EPS, residual=r, mx=m) for m in ("rows", "atoms"))
    h = x.double() + r.double()
    v = h * (h.square().mean(1, keepdim=True) + EPS) ** -0.5 * w.double()
    for out in (rows, atoms):
        assert _rounds_to(out["y"], v, 80 * U * v.abs())
        assert torch.equal(out["residual"], (x.float() + r.float()).to(torch.bfloat16))
    amax = v.view(T, d // 32, 32).abs().amax(2)
    place = torch.log2(amax / 448.0)
    got = rows["scales"].double() - 127
    edge = (place - place.round()).abs() < 1e-4
    assert ((got == place.ceil()) | (edge & ((got - place.ceil()).abs() <= 1))).all()
    scale = torch.exp2(got).repeat_interleave(32, 1)
    q = rows["codes"].view(torch.float8_e4m3fn).double() * scale
    assert ((q - v).abs() <= (2.0 ** -4 + 80 * U) * v.abs() + 2.0 ** -10 * scale * 1.001).all()
    assert torch.equal(rows["codes"], atoms["codes"])
    tiles = atoms["scales"].view(-1, d // 128, 32, 4, 4)                    # tile, K block, r0, r1, byte
    flat = tiles.permute(0, 3, 2, 1, 4).reshape(-1, d // 32)                # row = 32 r1 + r0
    assert torch.equal(flat[:T], rows["scales"]) and (flat[T:] == 0).all()


def test_passes_in_a_row_repeat_themselves():
    """The same inputs before and after another pass, nothing waited for in between."""
    ensure_lib()
    T, d = 4099, 7168
    one, two = ((_rows(T, d, torch.bfloat16, i), _rows(T, d, torch.bfloat16, i + 1, 4.0)) for i in (20, 30))
    w = _weight(d, torch.bfloat16, 40)
    a = mok.rms_norm(one[0], w, EPS, residual=one[1], mx="rows")
    mok.rms_norm(two[0], w, EPS, residual=two[1], mx="rows")
    b = mok.rms_norm(one[0], w, EPS, residual=one[1], mx="rows")
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_in_a_captured_graph():
    ensure_lib()
    T, d = 701, 1544
    x, r, w = _rows(T, d, torch.bfloat16, 50), _rows(T, d, torch.float32, 51), _weight(d, torch.float32, 52)
    ws = torch.zeros(mok.rms_norm_workspace_size(T, d), dtype=torch.uint8, device="cuda")

    def both():
        n = mok.rms_norm(x, w, EPS, residual=r)
        return {**n, **mok.rms_norm_backward(n["y"], n["residual"], w, EPS, dres=r, ws=ws)}

    want = both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(2):
        for t in got.values():
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(want[k], got[k]) for k in want)
