"""Gradient norm and AdamW (states in 32 and in 8 bits) against 64 bits.

Tolerances.  u = 2^-24.  m and v are two products and a sum: 4 u of the terms' magnitudes.  The
update is a product, a root, a sum, a quotient (8 u) of m and v, then w - lr (update + decay w):
u of w for each of the last two roundings.  The norm's sums carry less than 1e-5 in the worst case.
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
SIZES = [1, 7, 8, 31, 32, 33, 100, 4095, 4096, 4097, 12345, 0, 70001]
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _randn(n, seed, std=1.0, dtype=torch.float32):
    return (torch.randn(n, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


@pytest.mark.parametrize("sizes", [[], [0], [1], [5, 0, 9], SIZES, [3] * 1500, [1 << 22, 17]])
def test_grad_norm(sizes):
    ensure_lib()
    grads = [_randn(n, i, 0.1, TYPES["f32" if i % 3 == 0 else "bf16"]) for i, n in enumerate(sizes)]
    want = np.sqrt(sum((f64(g) ** 2).sum() for g in grads))
    for limit in (0.0, 0.5 * want, 2.0 * want):
        out = mok.grad_norm(grads, float(limit))
        assert abs(float(out[0]) - want) <= 1e-5 * want
        factor = 1.0 if limit == 0.0 or want == 0 else min(1.0, limit / want)
        assert abs(float(out[1]) - factor) <= 1e-5
        assert torch.equal(out, mok.grad_norm(mok.TensorList(grads), float(limit)))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_grad_norm_not_finite(bad):
    ensure_lib()
    grads = [_randn(50, 1), _randn(5000, 2, 1.0, torch.bfloat16)]
    grads[1][4999] = bad
    out = mok.grad_norm(grads, 1.0)
    assert not out[0].isfinite() and out[1].isnan()


def test_grad_norm_beyond_32_bits():
    ensure_lib()
    n = (1 << 32) + 1001
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-3:] = torch.tensor([3.0, 4.0, 12.0], device="cuda")
    assert float(mok.grad_norm([g], 0.0)[0]) == 13.0


def _weights(sizes, seed=100):
    params = [_randn(n, seed + i, 0.05, TYPES["f32" if i % 4 == 1 else "bf16"]) for i, n in enumerate(sizes)]
    grads = [_randn(n, seed + 50 + i, 0.01, TYPES["f32" if i % 3 == 0 else "bf16"]) for i, n in enumerate(sizes)]
    return params, grads, [0.1 if i % 2 else 0.0 for i in range(len(sizes))]


@pytest.mark.parametrize("sizes", [[], [0], [1], SIZES, [40, 3] * 300])
@pytest.mark.parametrize("clipped", [False, True])
def test_adamw_f32(sizes, clipped):
    ensure_lib()
    params, grads, decay = _weights(sizes)
    opt = mok.AdamW(params, betas=BETAS, eps=EPS, weight_decay=decay)
    w = [f64(opt.state["master"][i] if opt.state["master"][i] is not None else p) for i, p in enumerate(params)]
    m, v = [np.zeros_like(a) for a in w], [np.zeros_like(a) for a in w]
    lr = 3e-3
    for step in range(1, 4):
        clip = mok.grad_norm(grads, 0.25) if clipped else None
        factor = float(clip[1]) if clipped else 1.0
        opt.step(grads, lr, clip=clip)
        for i, g in enumerate(grads):
            start = w[i]
            w[i], m[i], v[i] = plain.adamw(w[i], f64(g) * factor, m[i], v[i], lr, *BETAS, EPS, decay[i], step)
            full = opt.state["master"][i] if params[i].dtype == torch.bfloat16 else params[i]
            size = lr * (np.abs(w[i] - start) / lr + 1.0)
            assert (np.abs(f64(full) - w[i]) <= step * (4 * U * np.abs(start) + 64 * U * size) + 1e-30).all()
            assert (np.abs(f64(opt.state["exp_avg"][i]) - m[i]) <= step * 8 * U * np.abs(f64(g)) + 1e-30).all()
            assert (np.abs(f64(opt.state["exp_avg_sq"][i]) - v[i]) <= step * 8 * U * f64(g) ** 2 + 1e-30).all()
            if params[i].dtype == torch.bfloat16:
                assert torch.equal(params[i], full.to(torch.bfloat16))
    assert opt.steps == 3


def _fraction(x, scale):
    """Lower neighbour of |x| on the E4M3 grid times scale, the grid's step there, the place."""
    q = np.abs(x) / scale
    with np.errstate(divide="ignore"):
        e = np.clip(np.floor(np.log2(np.maximum(q, 1e-300))), -6, 8)
    step = 2.0 ** (e - 3)
    low = np.floor(q / step) * step
    return low, step, (q - low) / step


@pytest.mark.parametrize("n", [1, 31, 32, 33, 4100, 9999])
def test_adamw_mxfp8_codes(n):
    """One step: scales from the block's amax, and every code the neighbour that the dither names."""
    ensure_lib()
    g = _randn(n, 7, 1e-2)
    g[::5] *= 1e-4                                   # a wide range inside a block
    if n > 100:
        g[64:96] = 0                                 # a block of zeros
    p = _randn(n, 8, 0.05, torch.bfloat16)
    opt = mok.AdamW([p], betas=BETAS, eps=EPS, states="mxfp8")
    master = f64(opt.state["master"][0])
    step, lr = 1, 1e-3
    opt.step([g], lr)
    w, m, v = plain.adamw(master, f64(g), 0 * master, 0 * master, lr, *BETAS, EPS, 0.0, step)
    assert (np.abs(f64(opt.state["master"][0]) - w) <= 4 * U * np.abs(master) + 64 * U * lr).all()
    pad = (-n) % 32
    low32 = np.uint64(0xFFFFFFFF)
    h = (np.uint64(0x85EBCA6B) * np.arange(n, dtype=np.uint64) + np.uint64(0x9E3779B9 * step)) & low32
    h = ((h ^ (h >> np.uint64(15))) * np.uint64(0x2C1B3C6D)) & low32
    h = ((h ^ (h >> np.uint64(12))) * np.uint64(0x297A2D39)) & low32
    h = h ^ (h >> np.uint64(15))
    for key, x, half, floor in (("exp_avg", m, h >> np.uint64(16), False), ("exp_avg_sq", v, h & np.uint64(0xFFFF), True)):
        s, amax = plain.mx_exponents(np.pad(x, (0, pad)))
        got = opt.state[key + "_scale"][0].cpu().numpy().astype(np.int64) - 127
        near = np.abs(amax / 448.0 * 2.0 ** -np.maximum(s, -126) - 1) < 1e-5
        assert ((got == s) | near).all()
        scale = np.repeat(2.0 ** got, 32)[:n]
        low, unit, place = _fraction(x, scale)
        r = (half + 0.5) / 2.0 ** 16
        want = low + unit * np.floor(place + r)
        if floor:
            want = np.where(x > 0, np.maximum(want, 2.0 ** -9), want)
        want = np.minimum(want, 448.0)
        q = plain.e4m3(opt.state[key][0].cpu().numpy())
        edge = np.abs(place + r - np.round(place + r)) < 1e-3    # fp32 arithmetic, 20 bits of mantissa
        assert (np.abs(q) == want)[~edge].all()
        assert (np.abs(np.abs(q) - want) <= unit * 1.001).all()
        assert (np.sign(q) == np.sign(x))[q != 0].all()
        if floor:
            assert (q[x > 0] > 0).all()


def test_adamw_mxfp8_averages_move():
    """With no gradient, 200 steps at beta2 = 0.999 shrink v to 0.8187 of its start and at beta1 =
    0.95 m to nothing; rounding to the nearest code would leave v where it was.  The mean over
    40000 elements deviates by at most 1% (dither noise of 10-20% per element, averaged)."""
    ensure_lib()
    n = 40000
    p, g = _randn(n, 9, 0.05), _randn(n, 10, 1e-2)
    opt = mok.AdamW([p], betas=(0.95, 0.999), eps=EPS, states="mxfp8")
    opt.step([g], 0.0)

    def mean_v():
        s = 2.0 ** (opt.state["exp_avg_sq_scale"][0].cpu().numpy().astype(np.float64) - 127)
        return (plain.e4m3(opt.state["exp_avg_sq"][0].cpu().numpy()) * np.repeat(s, 32)[:n]).mean()

    start = mean_v()
    assert abs(start / (1e-3 * (f64(g) ** 2).mean()) - 1) < 0.01
    zero = torch.zeros_like(g)
    for _ in range(200):
        opt.step([zero], 0.0)
    assert abs(mean_v() / start / 0.999 ** 200 - 1) < 0.01
    s = 2.0 ** (opt.state["exp_avg_scale"][0].cpu().numpy().astype(np.float64) - 127)
    m = plain.e4m3(opt.state["exp_avg"][0].cpu().numpy()) * np.repeat(s, 32)[:n]
    assert np.abs(m).mean() < 1e-3 * 0.05 * np.abs(f64(g)).mean()


@pytest.mark.parametrize("states", ["f32", "mxfp8"])
def test_adamw_many_tensors_equal_one_at_a_time(states):
    """800 tensors (three launches) give the bits of single calls; state buffers can be handed over."""
    ensure_lib()
    params, grads, _ = _weights([37, 64, 500, 1] * 200)
    alone = [p.clone() for p in params]
    opt = mok.AdamW(params, states=states)
    opt.step(grads, 1e-2)
    resumed = mok.AdamW(params, **opt.state_dict())
    resumed.step(mok.TensorList(grads), 1e-2)
    assert resumed.steps == 2
    for i in range(0, 800, 37):
        one = mok.AdamW([alone[i]], states=states)
        one.step([grads[i]], 1e-2)
        one.step([grads[i]], 1e-2)
        assert torch.equal(alone[i], params[i])
        for key in opt.state:
            if opt.state[key][i] is not None:
                assert torch.equal(one.state[key][0], opt.state[key][i]), key


@pytest.mark.parametrize("states", ["f32", "mxfp8"])
def test_adamw_skips_a_step_without_a_finite_norm(states):
    ensure_lib()
    params, grads, _ = _weights([100, 4097])
    opt = mok.AdamW(params, states=states)
    opt.step(grads, 1e-2, clip=mok.grad_norm(grads, 1.0))
    before = [p.clone() for p in params] + [t.clone() for v in opt.state.values() for t in v if t is not None]
    grads[1][5] = float("nan")
    opt.step(grads, 1e-2, clip=mok.grad_norm(grads, 1.0))
    after = params + [t for v in opt.state.values() for t in v if t is not None]
    assert all(torch.equal(a, b) for a, b in zip(before, after))


def test_adamw_refusals():
    ensure_lib()
    params, grads, _ = _weights([100, 33])
    opt = mok.AdamW(params, states="mxfp8")
    for bad in (grads[:1], [grads[0], grads[1][:32]], [grads[0], grads[1].half()], [grads[0].cpu(), grads[1]]):
        with pytest.raises(ValueError):
            opt.step(bad, 1e-3)
    with pytest.raises(ValueError):
        opt.step(grads, 1e-3, clip=torch.ones(1, device="cuda"))
    with pytest.raises(mok.MokError):
        opt.step(grads, float("nan"))
    assert opt.steps == 0
    state = opt.state_dict()["state"]
    for key, value in (("exp_avg", state["exp_avg"][:1]), ("exp_avg_sq", [state["exp_avg_sq"][0].float()] * 2),
                       ("exp_avg_scale", [None, None])):
        with pytest.raises(ValueError):
            mok.AdamW(params, states="mxfp8", state=dict(state, **{key: value}))
    with pytest.raises(ValueError):
        mok.AdamW(params, weight_decay=[0.1])
    with pytest.raises(ValueError):
        mok.TensorList([grads[0], torch.ones((4, 4), device="cuda").t()])
    with pytest.raises(ValueError):
        mok.grad_norm(grads, 1.0, ws=torch.zeros(4096, device="cuda"))
    with pytest.raises(mok.MokError):
        mok.grad_norm(grads, 1.0, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(mok.MokError):       # not 16-byte aligned
        mok.grad_norm([torch.ones(9, device="cuda")[1:]], 1.0)


def test_side_stream():
    """Both on a stream of their own, waiting for the inputs there."""
    ensure_lib()
    params, grads, _ = _weights([5000, 77])
    other = [p.clone() for p in params]
    opt, twin = mok.AdamW(params), mok.AdamW(other)
    clip = mok.grad_norm(grads, 0.1)
    opt.step(grads, 1e-2, clip=clip)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = mok.grad_norm(grads, 0.1)
        twin.step(grads, 1e-2, clip=again)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(clip, again) and all(torch.equal(p, q) for p, q in zip(params, other))


def test_adamw_beyond_32_bits():
    """More than 2^31 elements (17 GB on the device): the last ones get the step of a small tensor."""
    ensure_lib()
    n, tail = (1 << 31) + 4096 + 40, 40
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p[-tail:], g[-tail:] = _randn(tail, 1), _randn(tail, 2, 1.0, torch.bfloat16)
    q, h = p[-tail:].clone(), g[-tail:].clone()
    big, small = mok.AdamW([p], states="mxfp8"), mok.AdamW([q], states="mxfp8")
    big.step([g], 1e-2)
    small.step([h], 1e-2)
    assert torch.equal(p[-tail:], q) and (p[:-tail] == 0).all()
    assert torch.equal(big.state["exp_avg_scale"][0][-2:], small.state["exp_avg_scale"][0])
    assert (big.state["exp_avg"][0][:-tail] == 0).all()
