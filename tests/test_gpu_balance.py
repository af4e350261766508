"""Balance loss, z loss, counts and the logits' gradient against 64 bits.

Tolerances.  u = 2^-24.  A softmax entry carries the exponential's 2 ulp plus u |l - max|, its sum
over at most 512 terms and the division: below 64 u for |l - max| <= 30.  The gradient
p (a (c - <c,p>) + b lse) is compared relative to p (a (c + <c,p>) + b |lse|), the loss relative to
itself (all of its terms are positive); both with 256 u.
"""

import numpy as np
import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests import _around as plain
from tests._helpers import ensure_lib, f64

pytestmark = pytest.mark.gpu

TOL = 256 * 2.0 ** -24


def _inputs(T, E, k, seed, skew=1.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((T, E), generator=g) * 2 - skew * torch.log(torch.randperm(E, generator=g).float() + 1)
    return logits, logits.topk(k, dim=1).indices.to(torch.int32)


def _run(logits, idx, alpha, z, offsets=None, mask=None, **kw):
    T, E = logits.shape
    D = mok.dims(T, 128, E, idx.shape[1], 128, 0, 0)
    S = 1 if offsets is None else len(offsets) - 1
    ws = torch.zeros(mok.balance_loss_workspace_size(D, S), dtype=torch.uint8, device="cuda")
    out = mok.balance_loss(D, logits.cuda(), idx.cuda(), ws, alpha, z_coef=z,
                           seq_offsets=None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda(),
                           token_mask=None if mask is None else torch.from_numpy(mask).cuda(), **kw)
    return out, mok.read_status(ws)


def _check(logits, idx, alpha, z, offsets=None, mask=None):
    out, status = _run(logits, idx, alpha, z, offsets, mask)
    assert status == 0
    T, E = logits.shape
    S = 1 if offsets is None else len(offsets) - 1
    seq = plain.sequences(T, offsets, mask)
    loss, counts, dl = plain.balance(f64(logits), idx.numpy(), S, seq, alpha, z)
    assert (out["counts"].cpu().numpy() == counts).all()
    got = f64(out["loss"])
    assert (np.abs(got - loss) <= TOL * np.abs(loss)).all(), (got, loss)
    ok = seq >= 0
    n, n_seq = max(1, ok.sum()), np.bincount(seq[ok], minlength=S)
    L = f64(logits)
    p = np.exp(L - L.max(1, keepdims=True))
    lse = L.max(1) + np.log(p.sum(1))
    p /= p.sum(1, keepdims=True)
    c = counts[np.maximum(seq, 0)]
    a = np.where(ok, alpha * E / (idx.shape[1] * n * np.maximum(n_seq, 1)[np.maximum(seq, 0)]), 0)
    size = p * (a[:, None] * (c + (c * p).sum(1, keepdims=True)) + 2 * z / n * np.abs(lse)[:, None])
    assert (np.abs(f64(out["dlogits"]) - dl) <= TOL * size + 1e-30).all()
    assert (out["dlogits"].cpu().numpy()[~ok] == 0).all()
    again, _ = _run(logits, idx, alpha, z, offsets, mask)
    assert all(torch.equal(out[key], again[key]) for key in out)
    return out


@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (1, 512, 8), (7, 8, 8), (255, 16, 3), (256, 8, 2), (777, 40, 4),
                                   (300, 256, 8), (129, 384, 8), (64, 512, 5), (4097, 24, 2)])
@pytest.mark.parametrize("z", [0.0, 1e-3])
def test_one_sequence(T, E, k, z):
    ensure_lib()
    _check(*_inputs(T, E, k, T + E), 1e-2, z)


@pytest.mark.parametrize("T,E,k,S", [(50, 8, 2, 50), (400, 24, 3, 7), (1000, 256, 8, 5), (513, 384, 4, 100),
                                     (3000, 64, 8, 700), (3000, 16, 2, 2500), (6000, 24, 4, 3)])
def test_packed_and_masked(T, E, k, S):
    """Ragged sequences, some empty, tokens before the first and after the last, masked tokens."""
    ensure_lib()
    rng = np.random.default_rng(T)
    cuts = np.sort(rng.integers(T // 10, T - T // 10, S + 1)).tolist()
    cuts[-1] = max(cuts[-1], cuts[-2])
    logits, idx = _inputs(T, E, k, S)
    _check(logits, idx, 0.02, 1e-3, cuts, rng.random(T) < 0.7)
    _check(logits, idx, 0.02, 0.0, [0] + cuts[1:-1] + [T], None)


@pytest.mark.parametrize("k", [4, 8])
def test_selection_that_is_not_16_byte_aligned(k):
    ensure_lib()
    logits, idx = _inputs(900, 32, k, 12)
    D = mok.dims(900, 128, 32, k, 128, 0, 0)
    ws = torch.zeros(mok.balance_loss_workspace_size(D), dtype=torch.uint8, device="cuda")
    shifted = torch.empty(900 * k + 2, dtype=torch.int32, device="cuda")[2:].view(900, k)
    shifted.copy_(idx)
    want, _ = _run(logits, idx, 0.02, 1e-3)
    got = mok.balance_loss(D, logits.cuda(), shifted, ws, 0.02, z_coef=1e-3)
    assert all(torch.equal(want[key], got[key]) for key in want)
    with pytest.raises(mok.MokError):
        moved = torch.empty(900 * 32 + 1, device="cuda")[1:].view(900, 32)
        mok.balance_loss(D, moved, shifted, ws, 0.02)


def test_everything_masked():
    ensure_lib()
    logits, idx = _inputs(40, 16, 2, 1)
    out = _check(logits, idx, 0.02, 1e-3, [0, 0, 40, 40], np.zeros(40, dtype=bool))
    assert (out["loss"] == 0).all() and (out["counts"] == 0).all() and (out["dlogits"] == 0).all()


def test_masked_places_hold_anything():
    """NaN and inf in the logits of left-out tokens, and nonsense in their selection, change nothing."""
    ensure_lib()
    logits, idx = _inputs(200, 32, 4, 2)
    mask = np.random.default_rng(3).random(200) < 0.6
    want, _ = _run(logits, idx, 0.02, 1e-3, [0, 90, 200], mask)
    dirty, bad = logits.clone(), idx.clone()
    out_of = torch.from_numpy(~mask)
    dirty[out_of] = torch.tensor([float("nan"), float("inf")]).repeat(16)
    bad[out_of] = 10 ** 6
    got, status = _run(dirty, bad, 0.02, 1e-3, [0, 90, 200], mask)
    assert status == 0 and all(torch.equal(want[key], got[key]) for key in want)


def test_masked_experts():
    """-inf logits: probability and gradient 0; a token with nothing but -inf gives nothing; the
    type's lowest value is an ordinary, very small probability."""
    ensure_lib()
    logits, idx = _inputs(100, 24, 2, 4)
    logits[:, 5] = float("-inf")
    logits[:, 6] = torch.finfo(torch.float32).min
    idx = logits.topk(2, dim=1).indices.to(torch.int32)
    out, _ = _run(logits, idx, 0.02, 1e-3)
    loss, counts, dl = plain.balance(f64(logits), idx.numpy(), 1, np.zeros(100, dtype=np.int64), 0.02, 1e-3)
    assert (out["dlogits"][:, 5:7] == 0).all()
    assert np.abs(f64(out["loss"]) - loss).max() <= TOL * loss.max()
    assert np.abs(f64(out["dlogits"]) - dl).max() <= TOL * np.abs(dl).max()
    logits[7] = float("-inf")
    out, _ = _run(logits, idx, 0.02, 1e-3)
    assert (out["dlogits"][7] == 0).all() and out["loss"].isfinite().all()
    logits[8, 3] = float("nan")
    out, _ = _run(logits, idx, 0.02, 1e-3)
    assert out["dlogits"][8].isnan().any() and out["dlogits"][9].isfinite().all() and out["loss"].isnan().all()


def test_index_out_of_range_is_reported():
    ensure_lib()
    logits, idx = _inputs(64, 16, 2, 5)
    idx[3, 1], idx[9, 0] = 16, -1
    out, status = _run(logits, idx, 0.02, 0.0)
    assert status == -6
    _, counts, _ = plain.balance(f64(logits), idx.numpy(), 1, np.zeros(64, dtype=np.int64), 0.02, 0.0)
    assert (out["counts"].cpu().numpy() == counts).all()


def test_no_tokens():
    ensure_lib()
    out, status = _run(torch.empty((0, 16)), torch.empty((0, 2), dtype=torch.int32), 0.02, 1e-3)
    assert status == 0 and (out["loss"] == 0).all() and (out["counts"] == 0).all() and out["dlogits"].shape == (0, 16)


def test_on_the_layers_own_workspace_and_in_a_graph():
    """The layer's forward workspace will do; a captured graph replays the two launches."""
    ensure_lib()
    logits, idx = _inputs(700, 64, 4, 11)
    D = mok.dims(700, 128, 64, 4, 128, 0, 0)
    ws = torch.zeros(mok.workspace_size(D), dtype=torch.uint8, device="cuda")
    want, _ = _run(logits, idx, 0.02, 1e-3)
    lc, ic = logits.cuda(), idx.cuda()
    got = mok.balance_loss(D, lc, ic, ws, 0.02, z_coef=1e-3)
    assert all(torch.equal(want[key], got[key]) for key in want) and mok.read_status(ws) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mok.balance_loss(D, lc, ic, ws, 0.02, z_coef=1e-3)
    for _ in range(3):
        for t in got.values():
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(want[key], got[key]) for key in want)


def test_upstream_gradient_and_no_gradient():
    ensure_lib()
    logits, idx = _inputs(90, 16, 2, 6)
    one, _ = _run(logits, idx, 0.02, 1e-3)
    four, _ = _run(logits, idx, 0.02, 1e-3, grad=torch.tensor([4.0], device="cuda"))
    assert torch.equal(four["dlogits"], 4 * one["dlogits"]) and torch.equal(four["loss"], one["loss"])
    none, _ = _run(logits, idx, 0.02, 1e-3, want_dlogits=False)
    assert "dlogits" not in none and torch.equal(none["loss"], one["loss"])


def test_gradient_against_differences():
    ensure_lib()
    T, E, k = 60, 16, 3
    logits, idx = _inputs(T, E, k, 7)
    seq = plain.sequences(T, [0, 10, 10, 45, 60], np.random.default_rng(8).random(T) < 0.8)
    out, _ = _run(logits, idx, 0.5, 0.1, [0, 10, 10, 45, 60], seq >= 0)
    u = np.random.default_rng(9).standard_normal((T, E))
    f = lambda t: plain.balance(f64(logits) + t * u, idx.numpy(), 4, seq, 0.5, 0.1)[0].sum()  # noqa: E731
    want = (f(1e-5) - f(-1e-5)) / 2e-5
    got = (f64(out["dlogits"]) * u).sum()
    assert abs(got - want) <= 1e-5 * np.abs(f64(out["dlogits"]) * u).sum()


def test_offsets_beyond_32_bits():
    """T E > 2^31 (17 GB on the device): the last tokens' gradients."""
    ensure_lib()
    T, E, k = (1 << 22) + 9, 512, 1
    tail, tail_idx = _inputs(9, E, k, 10)
    D = mok.dims(T, 128, E, k, 128, 0, 0)
    logits = torch.zeros((T, E), device="cuda")
    idx = (torch.arange(T, device="cuda") % E).to(torch.int32).unsqueeze(1)
    logits[-9:], idx[-9:] = tail.cuda(), tail_idx.cuda()
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    mask[-9:] = True
    ws = torch.zeros(mok.balance_loss_workspace_size(D), dtype=torch.uint8, device="cuda")
    out = mok.balance_loss(D, logits, idx, ws, 0.02, z_coef=1e-3, token_mask=mask)
    loss, counts, dl = plain.balance(f64(tail), tail_idx.numpy(), 1, np.zeros(9, dtype=np.int64), 0.02, 1e-3)
    assert (out["counts"].cpu().numpy() == counts).all()
    assert np.abs(f64(out["loss"]) - loss).max() <= TOL * loss.max()
    assert np.abs(f64(out["dlogits"][-9:]) - dl).max() <= TOL * np.abs(dl).max()
    assert (out["dlogits"][:-9] == 0).all()
