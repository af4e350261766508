"""Balance and z loss over the whole range of fp32 logits, and where a warp takes many tokens.

Tolerances.  u = 2^-24.  A softmax entry carries two roundings of its exponent, at most 2 u |l - max|
<= 60 u for |l - max| <= 30, the exponential's 2 ulp, the sum over at most 512 terms (lanes, then 5
shuffles: 21 u) and the division: below 96 u.  The gradient p (a (c - <c,p>) + b lse) is compared
relative to p (a (c + <c,p>) + b |lse|), with 256 u.  The losses are sums of terms of one sign: a
warp adds at most T / 2000 + 1 of them, then 8 warps, 4 per thread and 5 + 8 more: 256 u too.
"""

import numpy as np
import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests._helpers import ensure_lib

pytestmark = pytest.mark.gpu

TOL = 256 * 2.0 ** -24
LOWEST = torch.finfo(torch.float32).min


def _logits(T, E, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = 2 * torch.randn((T, E), generator=g, device="cuda") - torch.log(1.0 + torch.arange(E, device="cuda"))
    return logits, logits.topk(k, dim=1).indices.to(torch.int32)


def _run(logits, idx, alpha, z, offsets=None, mask=None):
    T, E = logits.shape
    S = 1 if offsets is None else offsets.numel() - 1
    D = mok.dims(T, 128, E, idx.shape[1], 128, 0, 0)
    ws = torch.zeros(mok.balance_loss_workspace_size(D, S), dtype=torch.uint8, device="cuda")
    out = mok.balance_loss(D, logits, idx, ws, alpha, z_coef=z, seq_offsets=offsets, token_mask=mask)
    assert mok.read_status(ws) == 0
    return out


def _plain(logits, idx, alpha, z, offsets=None, mask=None):
    """loss [2], counts, dlogits and the size that the gradient's error is relative to, in 64 bits."""
    (T, E), k = logits.shape, idx.shape[1]
    S = 1 if offsets is None else offsets.numel() - 1
    ok = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask.clone()
    t = torch.arange(T, device="cuda")
    seq = torch.zeros(T, dtype=torch.long, device="cuda")
    if offsets is not None:
        seq = torch.bucketize(t, offsets.long(), right=True) - 1
        ok &= (seq >= 0) & (seq < S)
        seq = seq.clamp(0, S - 1)
    chosen = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, idx.long(), 1.0) * ok.unsqueeze(1)
    counts = torch.zeros((S, E), dtype=torch.float64, device="cuda").index_add_(0, seq, chosen)
    n, n_seq = max(1, int(ok.sum())), torch.bincount(seq[ok], minlength=S).clamp(min=1)
    l = logits.double()
    lse = torch.logsumexp(l, 1)
    p = torch.softmax(l, 1)      # not exp(l - lse): log E is lost beside 1e20 in 64 bits too
    c = counts[seq]
    inner = (c * p).sum(1)
    a = ok * (alpha * E / k / n) / n_seq[seq]
    b = ok * (2.0 * z / n)
    loss = torch.stack([(a * inner).sum(), (0.5 * b * lse * lse).sum()])
    dl = p * (a.unsqueeze(1) * (c - inner.unsqueeze(1)) + (b * lse).unsqueeze(1))
    size = p * (a.unsqueeze(1) * (c + inner.unsqueeze(1)) + (b * lse.abs()).unsqueeze(1))
    return loss, counts, dl, size


HUGE = [LOWEST, -1e20, -4e9, 4e9, 1e20, 3e38]


@pytest.mark.parametrize("value", HUGE)
@pytest.mark.parametrize("z", [0.0, 1e-3])
def test_rows_of_one_huge_value(value, z):
    """A row whose mask leaves nothing (every logit the type's lowest value) and rows of other huge
    finite values have the uniform softmax and touch no other row."""
    ensure_lib()
    logits, idx = _logits(70, 40, 3, 1)
    clean = _run(logits, idx, 0.02, z)
    logits[11] = value
    out = _run(logits, idx, 0.02, z)
    loss, counts, dl, size = _plain(logits, idx, 0.02, z)
    assert torch.equal(out["counts"].double(), counts)
    assert abs(float(out["loss"][0]) - float(loss[0])) <= TOL * float(loss[0])
    assert ((out["dlogits"].double() - dl).abs() <= TOL * size + 1e-30).all()
    others = torch.arange(70, device="cuda") != 11
    assert torch.equal(out["dlogits"][others], clean["dlogits"][others])


@pytest.mark.parametrize("z", [0.0, 1e-3])
def test_one_huge_logit(z):
    """One expert takes all of a row; the distance to the others may overflow."""
    ensure_lib()
    logits, idx = _logits(70, 40, 3, 2)
    logits[11, 5], logits[12, 5], logits[12, 6:] = 3e38, 3e38, LOWEST
    out = _run(logits, idx, 0.02, z)
    loss, counts, dl, size = _plain(logits, idx, 0.02, z)
    assert abs(float(out["loss"][0]) - float(loss[0])) <= TOL * float(loss[0])
    assert ((out["dlogits"].double() - dl).abs() <= TOL * size + 1e-30).all()


@pytest.mark.parametrize("value", HUGE)
@pytest.mark.parametrize("z", [0.0, 1e-3])
def test_z_loss_of_huge_logits(value, z):
    """Zero when it is off, the value wherever fp32 holds it, though log-sum-exp squared overflows."""
    ensure_lib()
    logits, idx = _logits(50, 16, 2, 3)
    logits[7] = value
    got = float(_run(logits, idx, 0.02, z)["loss"][1])
    want = float(_plain(logits, idx, 0.02, z)[0][1])
    if want > torch.finfo(torch.float32).max:
        assert got == float("inf")
    else:
        assert abs(got - want) <= TOL * want


@pytest.mark.parametrize("T,E,k", [(40001, 128, 8), (30011, 256, 4), (20011, 384, 8), (33333, 512, 5)])
@pytest.mark.parametrize("packed", [False, True])
def test_many_tokens_per_warp(T, E, k, packed):
    """Warps take 6 to 11 tokens each, so that every place of their ring is filled again, and
    sequences end within a warp's tokens; every row is compared."""
    ensure_lib()
    logits, idx = _logits(T, E, k, T)
    offsets = mask = None
    if packed:
        rng = np.random.default_rng(T)
        cuts = np.sort(rng.integers(3, T - 3, 301)).astype(np.int32)
        offsets = torch.from_numpy(cuts).cuda()
        mask = torch.from_numpy(rng.random(T) < 0.8).cuda()
    z = 1e-3 if packed else 0.0
    out = _run(logits, idx, 0.02, z, offsets, mask)
    loss, counts, dl, size = _plain(logits, idx, 0.02, z, offsets, mask)
    assert torch.equal(out["counts"].double(), counts)
    assert ((out["loss"].double() - loss).abs() <= TOL * loss.abs()).all()
    assert ((out["dlogits"].double() - dl).abs() <= TOL * size + 1e-30).all()
