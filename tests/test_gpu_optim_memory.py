"""AdamW refuses weights and states that share memory: a step would update them from several blocks."""

import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests._helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("states", ["f32", "mxfp8"])
def test_shared_memory_is_refused(states):
    ensure_lib()
    flat = torch.zeros(256, device="cuda")
    for params in ([flat, flat], [flat[:136], flat[128:]], [flat[64:72], flat], [flat[:8], flat[128:], flat[:1]]):
        with pytest.raises(ValueError, match="share memory"):
            mok.AdamW(params, states=states)
    state = mok.AdamW([flat], states=states).state_dict()["state"]
    with pytest.raises(ValueError, match="share memory"):
        mok.AdamW([flat], states=states, state=dict(state, exp_avg_sq=state["exp_avg"]))


@pytest.mark.parametrize("states", ["f32", "mxfp8"])
def test_neighbours_and_empty_tensors_are_fine(states):
    ensure_lib()
    flat = torch.zeros(256, device="cuda")
    params = [flat[128:], flat[64:64], flat[:64], flat[64:128]]
    opt = mok.AdamW(params, states=states)
    opt.step([torch.ones_like(p) for p in params], 1e-2)
    assert torch.allclose(flat, torch.full_like(flat, -1e-2), rtol=1e-5, atol=0)
    again = mok.AdamW(params, **opt.state_dict())
    assert again.steps == 1
