"""The training program's selection, norms on both sides and checkpoints: every weight that has a gradient moves
against it, and the balance bias moves towards experts with fewer tokens than the mean, by its rate."""

import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from mixture_experts_layer_14_gb300 import train_block
from tests._helpers import ensure_lib

pytestmark = pytest.mark.gpu


def _record(monkeypatch):
    """The blocks that the program makes, and what the trained one saw and gave step by step."""
    made = []

    class Recorded(mok.MoEBlock):
        def __init__(self, *args, **kw):
            super().__init__(*args, **kw)
            self.steps = []
            made.append(self)

        def gradients(self, g):
            out = super().gradients(g)
            names, params = self.parameters()
            bias = self.W.get("balance_bias")
            self.steps.append(dict(
                weights={n: p.clone() for n, p in zip(names, params)}, grads={n: v.clone() for n, v in zip(names, out)},
                bias=None if bias is None else bias.clone(), counts=self.aux["counts"].sum(0).double()))
            return out

    monkeypatch.setattr(train_block, "MoEBlock", Recorded)
    return made


CASES = [dict(scoring="sigmoid", post_norm=True, checkpoint="mxfp8"), dict(scoring="softmax", post_norm=True),
         dict(scoring="sigmoid", dtype="mxfp8", post_norm=True, checkpoint="mxfp8"), dict(post_norm=True, states="mxfp8"),
         dict(checkpoint="mxfp8")]


@pytest.mark.parametrize("kw", CASES)
def test_weights_and_balance_bias_move(monkeypatch, kw):
    ensure_lib()
    made = _record(monkeypatch)
    train_block.train(steps=3, lr=1e-2, bias_rate=0.25, **kw)
    block = made[-1]
    first, second, third = block.steps
    names, params = block.parameters()
    assert ("post_norm" in names and "post_gate" in names) == bool(kw.get("post_norm"))
    for n in names:
        step, g = second["weights"][n].double() - first["weights"][n].double(), first["grads"][n].double()
        assert torch.isfinite(g).all() and g.any(), n
        # The first step of AdamW is lr times the gradient's sign, where that is well above its epsilon; the
        # decay (1e-4 of the weight) and the rounding of a bf16 weight below 1/2 (2^-10) are smaller.
        big = (g.abs() > 0.1 * g.abs().max()) & ((first["weights"][n].double().abs() < 0.5) | (not n.startswith("W")))
        assert big.any() and (step[big] * g[big] < 0).all(), n
        assert not torch.equal(third["weights"][n], second["weights"][n]), n
    if "scoring" in kw:
        for a, b in ((first, second["bias"]), (second, third["bias"]), (third, block.W["balance_bias"])):
            want = a["bias"].double() + 0.25 * torch.sign(a["counts"].mean() - a["counts"])
            assert torch.equal(b.double(), want)  # quarters: exact
        assert (first["bias"] == 0).all() and second["bias"].any()
    else:
        assert block.W.get("balance_bias") is None
