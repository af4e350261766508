"""Choice of experts where scores saturate: keys that are equal in 64 bits go to the larger logit.

The reference order is that of the scores in 260 decimal digits (e^-400, the least one here, is 1e-174)."""

from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests._helpers import ensure_lib

pytestmark = pytest.mark.gpu

getcontext().prec = 260


def _keys(l, scoring, bias):
    v = [Decimal(float(x)) for x in l]
    if scoring == "sigmoid":
        s = [1 / (1 + (-x).exp()) for x in v]
    else:
        e = [(x - max(v)).exp() for x in v]
        s = [x / sum(e) for x in e]
    return [a + Decimal(float(b)) for a, b in zip(s, bias)]


def _choose(l, k, scoring, bias, groups, kept):
    c, n = _keys(l, scoring, bias), len(l) // groups
    best = sorted(range(groups), key=lambda g: (-max(c[g * n:g * n + n]), g))[:kept]
    return sorted((e for g in best for e in range(g * n, g * n + n)), key=lambda e: (-c[e], e))[:k]


def _run(l, k, scoring, bias, groups=1, kept=1):
    ensure_lib()
    D = mok.dims(len(l), 128, l.shape[1], k, 128, 0, 0)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sel = mok.Selection(scoring, n_groups=groups, topk_groups=kept)
    b = None if bias is None else torch.from_numpy(bias).cuda()
    idx, _ = mok.select_experts(D, sel, torch.from_numpy(l).cuda(), ws, bias=b)
    assert mok.read_status(ws) == 0
    return idx.cpu().tolist()


def test_two_saturated_scores():
    """1 / (1 + e^-40) and 1 / (1 + e^-50) are 1 in 64 bits."""
    l = np.full((1, 8), -1.0, dtype=np.float32)
    l[0, 2], l[0, 5] = 40.0, 50.0
    for bias in (None, np.zeros(8, dtype=np.float32), np.full(8, -3.0, dtype=np.float32)):
        assert _run(l, 2, "sigmoid", bias) == [[5, 2]]
        assert _run(l, 1, "sigmoid", bias, groups=2, kept=1) == [[5]]


@pytest.mark.parametrize("scoring,lo,hi", [("sigmoid", 38.0, 90.0), ("sigmoid", 20.0, 60.0), ("sigmoid", -60.0, -30.0),
                                           ("softmax", -400.0, 0.0)])
@pytest.mark.parametrize("E,k,groups,kept", [(16, 3, 1, 1), (64, 8, 1, 1), (256, 8, 1, 1), (64, 4, 8, 3), (256, 8, 8, 4)])
@pytest.mark.parametrize("bias", [0.0, 0.5])
def test_saturated_rows(scoring, lo, hi, E, k, groups, kept, bias):
    """One bias for all: the scores of most experts of a row vanish beside it, or beside 1."""
    rng = np.random.default_rng(E + k)
    l = rng.uniform(lo, hi, (24, E)).astype(np.float32)
    b = np.full(E, bias, dtype=np.float32)
    assert _run(l, k, scoring, b, groups, kept) == [_choose(r, k, scoring, b, groups, kept) for r in l]


@pytest.mark.parametrize("more", [False, True])
def test_biases_of_two_kinds(more):
    """Experts of either bias in the logits' order; the larger bias before the smaller one.  ``more``: more
    experts than lanes of a warp are equal in 64 bits."""
    rng = np.random.default_rng(5)
    E = 256 if more else 64
    l = rng.uniform(40.0, 80.0, (16, E)).astype(np.float32)
    b = np.where(np.arange(E) % 3 == 0, 0.25, 0.0).astype(np.float32)
    b[:E // 2] = 0.0
    assert _run(l, 8, "sigmoid", b) == [_choose(r, 8, "sigmoid", b, 1, 1) for r in l]


def test_equal_logits_still_go_to_the_lower_index():
    l = np.full((3, 64), 45.0, dtype=np.float32)
    l[1, 10:40] = 44.0
    l[2, 63] = 46.0
    assert _run(l, 4, "sigmoid", np.full(64, 0.5, dtype=np.float32)) == [[0, 1, 2, 3], [0, 1, 2, 3], [63, 0, 1, 2]]
