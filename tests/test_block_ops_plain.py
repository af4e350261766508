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
