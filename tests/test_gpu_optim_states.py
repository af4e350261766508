"""AdamW's 8-bit states on the path that carries most of the work, and how far the states hold.

Tolerances.  u = 2^-24.  As in the tests of single steps: 4 u of w and 64 u of lr for the master, and
codes exactly the neighbour that the dither names, except where the place between two codes is
within 1e-3 of a threshold (fp32 arithmetic, 20 bits of the place), plus 8 u of the sum's terms where
these cancel: there either neighbour will do.
"""

import numpy as np
import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests import _around as plain
from tests._helpers import ensure_lib, f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BETAS, EPS = (0.9, 0.95), 1e-8
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _randn(n, seed, std=1.0, dtype=torch.float32):
    return (torch.randn(n, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


def _values(opt, key, n):
    """A state in 64 bits, and its blocks' scales element by element."""
    s = np.repeat(2.0 ** (opt.state[key + "_scale"][0].cpu().numpy().astype(np.float64) - 127), 32)[:n]
    return plain.e4m3(opt.state[key][0].cpu().numpy()) * s, s


def _thresholds(n, step):
    """r of exp_avg and of exp_avg_sq for every element."""
    low32 = np.uint64(0xFFFFFFFF)
    h = (np.uint64(0x85EBCA6B) * np.arange(n, dtype=np.uint64) + np.uint64((0x9E3779B9 * step) & 0xFFFFFFFF)) & low32
    h = ((h ^ (h >> np.uint64(15))) * np.uint64(0x2C1B3C6D)) & low32
    h = ((h ^ (h >> np.uint64(12))) * np.uint64(0x297A2D39)) & low32
    h = h ^ (h >> np.uint64(15))
    return h >> np.uint64(16), h & np.uint64(0xFFFF)


@pytest.mark.parametrize("param", ["bf16", "f32"])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
def test_mxfp8_codes_of_whole_chunks(param, grad):
    """Three chunks of 8192 elements and a ragged one through three clipped steps: each step's codes,
    scales and weights follow from the states held before it."""
    ensure_lib()
    n, lr = 3 * 8192 + 33, 1e-3
    p = _randn(n, 1, 0.05, TYPES[param])
    opt = mok.AdamW([p], betas=BETAS, eps=EPS, weight_decay=0.1, states="mxfp8")
    for step in (1, 2, 3):
        g = _randn(n, 10 + step, 1e-2)
        g[::5] *= 1e-3                                   # a wide range inside a block
        g[64:96] = 0
        g = g.to(TYPES[grad])
        m, v = _values(opt, "exp_avg", n)[0], _values(opt, "exp_avg_sq", n)[0]
        master = opt.state["master"][0] if param == "bf16" else p
        start = f64(master)
        clip = mok.grad_norm([g], 0.5)
        opt.step([g], lr, clip=clip)
        factor = float(clip[1])
        assert factor < 0.8
        terms = BETAS[0] * np.abs(m) + (1 - BETAS[0]) * factor * np.abs(f64(g))   # m may cancel
        w, m, v = plain.adamw(start, f64(g) * factor, m, v, lr, *BETAS, EPS, 0.1, step)
        size = lr * (np.abs(w - start) / lr + 1.0)
        assert (np.abs(f64(master) - w) <= 4 * U * np.abs(start) + 64 * U * size).all()
        if param == "bf16":
            assert torch.equal(p, master.to(torch.bfloat16))
        for key, x, r, floor in zip(("exp_avg", "exp_avg_sq"), (m, v), _thresholds(n, step), (False, True)):
            got, scale = _values(opt, key, n)
            s, amax = plain.mx_exponents(np.pad(x, (0, -n % 32)))
            held = opt.state[key + "_scale"][0].cpu().numpy().astype(np.int64) - 127
            near = np.abs(amax / 448.0 * 2.0 ** -np.maximum(s, -126.0) - 1) < 1e-5
            assert ((held == s) | near).all()
            q = np.abs(x) / scale
            with np.errstate(divide="ignore"):
                e = np.clip(np.floor(np.log2(np.maximum(q, 1e-300))), -6, 8)
            unit = 2.0 ** (e - 3)
            place = q / unit - np.floor(q / unit) + (r + 0.5) / 2.0 ** 16
            want = np.minimum(unit * (np.floor(q / unit) + np.floor(place)), 448.0)
            if floor:
                want = np.where(x > 0, np.maximum(want, 2.0 ** -9), want)
            edge = np.abs(place - np.round(place)) < 1e-3 + 8 * U * (v if floor else terms) / (scale * unit)
            assert (np.abs(got / scale) == want)[~edge].all()
            assert (np.abs(np.abs(got / scale) - want) <= unit * 1.001).all()
            assert (np.sign(got) == np.sign(x))[got != 0].all()


def test_mxfp8_second_moment_has_a_lower_limit():
    """What the format promises of exp_avg_sq under constant gradients: the mean is the value where
    an element's gradients are 1/300 of its block's largest, and code 1 (2^-9 of the scale) where
    they are 1/3000.  The means over 2000 and 30000 elements deviate by at most 2%: an element wanders
    by 1.3 codes of 2.3 in the second case, which the mean divides by 170, and what the limit adds
    while the scale still grows (up to step 15) has shrunk by 0.95^105 after 120 steps."""
    ensure_lib()
    n = 32 * 2000
    g = torch.full((n // 32, 32), 1e-2 / 300, device="cuda")
    g[:, 16:], g[:, 0] = 1e-2 / 3000, 1e-2
    g = g.view(-1)
    p = torch.zeros(n, device="cuda")
    opt = mok.AdamW([p], betas=BETAS, eps=EPS, states="mxfp8")
    for _ in range(120):
        opt.step([g], 0.0)
    v, s = (a.reshape(-1, 32) for a in _values(opt, "exp_avg_sq", n))
    want = (1 - BETAS[1] ** 120) * f64(g).reshape(-1, 32) ** 2
    assert abs(v[:, 0].mean() / want[0, 0] - 1) < 0.02
    assert abs(v[:, 1:16].mean() / want[0, 1] - 1) < 0.02
    assert (v[:, 16:] == s[:, 16:] * 2.0 ** -9).all() and (v[:, 16:] > 20 * want[:, 16:]).all()


def test_in_a_captured_graph():
    """Norm and clipping from a replayed graph, on values that changed since the capture."""
    ensure_lib()
    sizes = [5000, 77, 0, 8193]
    grads = [_randn(n, i, 0.1, TYPES["f32" if i % 2 else "bf16"]) for i, n in enumerate(sizes)]
    params = [torch.zeros(n, device="cuda") for n in sizes]
    twins = [p.clone() for p in params]
    held = mok.TensorList(grads)
    ws = torch.zeros(mok.grad_norm_workspace_size(held), dtype=torch.uint8, device="cuda")
    opt, twin = mok.AdamW(params, states="mxfp8"), mok.AdamW(twins, states="mxfp8")
    mok.grad_norm(held, 0.3, ws=ws)                       # loads the kernels
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        clip = mok.grad_norm(held, 0.3, ws=ws)
        opt.step(held, 1e-2, clip=clip)
    for t in grads:
        t.mul_(2)
    graph.replay()
    want = mok.grad_norm(grads, 0.3)
    twin.step(grads, 1e-2, clip=want)
    torch.cuda.synchronize()
    assert torch.equal(clip, want) and all(torch.equal(a, b) for a, b in zip(params, twins))
