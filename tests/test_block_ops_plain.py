"""The plain forms of the block's operators against differences of themselves (no GPU)."""

import numpy as np
import pytest

from tests import _block


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_selection_gradient_against_differences(scoring, renorm):
    rng = np.random.default_rng(3)
    l = rng.normal(size=(5, 16))
    l[1, 3] = -np.inf
    idx, _ = _block.select(l, 4, scoring)
    dw = rng.normal(size=(5, 4))

    def loss(v):
        s = _block.scores(v, scoring)
        w = np.take_along_axis(s, idx, 1)
        w = w / w.sum(1, keepdims=True) if renorm else w
        return 1.7 * (w * dw).sum()

    got, h = _block.select_grad(l, idx, dw, scoring, renorm, 1.7), 1e-5
    for t in range(5):
        for e in range(16):
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((loss(a) - loss(b)) / (2 * h) - got[t, e]) < 1e-8


def test_selection_rules():
    """Groups, ties, experts that are shut off and biases, by hand."""
    l = np.array([[0.0, 1.0, 5.0, -9.0, 2.0, 2.0, 2.0, 2.0]])
    assert _block.select(l, 2, "sigmoid")[0].tolist() == [[2, 4]]
    # sums of two: (2, 2) beats (5, -9) and (0, 1)
    assert _block.select(l, 2, "sigmoid", groups=4, kept=1, by="top2")[0].tolist() == [[4, 5]]
    assert _block.select(l, 2, "sigmoid", groups=4, kept=1, by="max")[0].tolist() == [[2, 3]]
    bias = np.array([0, 0, -2.0, 0, 0, 0, 0, 0.5])
    idx, w = _block.select(l, 2, "sigmoid", bias=bias)
    assert idx.tolist() == [[7, 4]] and np.allclose(w, 0.5)
    l[0, :7] = -np.inf
    idx, w = _block.select(l, 3, "softmax")
    assert idx.tolist() == [[7, 0, 1]] and w.tolist() == [[1.0, 0.0, 0.0]]


@pytest.mark.parametrize("next_norm,gated", [(True, True), (True, False), (False, True)])
def test_sandwich_gradient_against_differences(next_norm, gated):
    rng = np.random.default_rng(4)
    T, d = 3, 8
    v = dict(x=rng.normal(size=(T, d)), r=rng.normal(size=(T, d)), post=rng.normal(size=d))
    if next_norm:
        v["weight"] = rng.normal(size=d)
    if gated:
        v["gate"], v["token_gate"] = rng.normal(size=d), rng.normal(size=T)
    dh, dv = rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def loss(**kw):
        h, y = _block.sandwich(**kw, a=0.7)
        return (h * dh).sum() + (0.0 if y is None else (y * dv).sum())

    h, _ = _block.sandwich(**v, a=0.7)
    rest = {k: v[k] for k in ("weight", "gate", "token_gate") if k in v}
    g = _block.sandwich_grad(v["x"], h, v["post"], dv if next_norm else None, dh, a=0.7, **rest)
    names = dict(x="dx", r="dresidual", post="dpost_weight", weight="dweight", gate="dgate", token_gate="dtoken_gate")
    for k in v:
        for i in np.ndindex(v[k].shape):
            lo, hi = v[k].copy(), v[k].copy()
            lo[i] -= 1e-5
            hi[i] += 1e-5
            diff = (loss(**dict(v, **{k: hi})) - loss(**dict(v, **{k: lo}))) / 2e-5
            assert abs(diff - g[names[k]][i]) < 1e-7
