"""Rows of the norms on both sides whose copies do not arrive, without a fault: the copies from one row on
are left out, their waits run out after a short limit, and these rows are NaN in every output, never what
was in shared memory before."""

import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests._helpers import ensure_lib

pytestmark = pytest.mark.gpu

NAN_CODE = 0x7f  # E4M3; 0xff is the other one


def _lost(t):
    """Which rows hold nothing but NaN."""
    m = (t & 0x7f) == NAN_CODE if t.dtype == torch.uint8 else t.isnan()
    return m.all(1)


def _make(T, d, res, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return dict(x=torch.randn((T, d), generator=g, device="cuda").bfloat16(),
                r=torch.randn((T, d), generator=g, device="cuda").to(torch.float32 if res == "f32" else torch.bfloat16),
                post=1 + 0.1 * torch.randn(d, generator=g, device="cuda"), w=1 + 0.1 * torch.randn(d, generator=g, device="cuda"))


# from the first, a middle and the last turn on; a row a warp's and a block's, one to four vectors per thread
CASES = [(5, 7168, "bf16", 2), (20011, 128, "f32", 7), (20011, 128, "bf16", 12345), (9001, 512, "bf16", 4000),
         (1300, 4096, "f32", 1299), (1100, 7168, "bf16", 700), (1301, 4480, "f32", 0), (400, 16384, "f32", 200)]


@pytest.mark.parametrize("T,d,res,first", CASES)
@pytest.mark.parametrize("next_norm", [True, False])
def test_forward(T, d, res, first, next_norm):
    ensure_lib()
    v = _make(T, d, res)
    args = dict(weight=v["w"], mx="rows" if d % 256 else "atoms", save="mxfp8") if next_norm else dict(save="mxfp8")
    clean = mok.sandwich_norm(v["x"], v["r"], v["post"], **args)
    mok.selftest_lost_rows(first)
    out = mok.sandwich_norm(v["x"], v["r"], v["post"], **args)
    torch.cuda.synchronize()
    for k in out:
        if k.endswith("scales"):
            if out[k].dim() == 2:
                assert torch.equal(out[k][:first], clean[k][:first]), k
            continue
        assert _lost(out[k][first:]).all(), k
        # a block that waits in vain for one row may give up its next; here every row before was fetched
        assert torch.equal(out[k][:first], clean[k][:first]), k
    again = mok.sandwich_norm(v["x"], v["r"], v["post"], **args)  # the next call is whole
    assert all(torch.equal(again[k], clean[k]) for k in clean)


def test_withdrawn_and_refused():
    L = ensure_lib()
    assert L.mok_selftest_lost_rows(-2, 1000) == -1 and L.mok_selftest_lost_rows(0, 0) == -1
    assert L.mok_selftest_lost_rows(0, 10**10) == -1
    v = _make(9, 256, "bf16")
    mok.selftest_lost_rows(3)
    mok.selftest_lost_rows(-1)
    assert not mok.sandwich_norm(v["x"], v["r"], v["post"])["residual"].isnan().any()


@pytest.mark.parametrize("T,d,res,first", CASES[:-1] + [(330, 8192, "bf16", 160), (400, 9216, "bf16", 155)])
@pytest.mark.parametrize("next_norm,dh,packed", [(True, True, False), (False, True, False), (True, False, True), (False, True, True)])
def test_backward(T, d, res, first, next_norm, dh, packed):
    """Lost rows are NaN in dx, dresidual and the token gate's gradient, and so are the weights' gradients;
    the status word says why."""
    ensure_lib()
    v = _make(T, d, res)
    dy, tg = _make(T, d, res, 4)["x"], torch.rand(T, device="cuda")
    x, h = (mok.activation_pack(v["x"]), mok.activation_pack(v["r"])) if packed else (v["x"], v["r"])
    ws = torch.zeros(mok.sandwich_norm_workspace_size(T, d), dtype=torch.uint8, device="cuda")

    def run():
        return mok.sandwich_norm_backward(
            x, h if next_norm else None, v["post"], dy=dy if next_norm else None, dres=v["r"] if dh else None,
            weight=v["w"] if next_norm else None, token_gate=tg, residual_dtype=v["r"].dtype, ws=ws)
    clean = run()
    assert mok.read_status(ws) == 0 and not any(t.isnan().any() for t in clean.values())
    mok.selftest_lost_rows(first)
    out = run()
    assert mok.read_status(ws) == -5  # MOK_ERR_TIMEOUT
    for k in ("dx", "dresidual", "dtoken_gate"):
        assert out[k][first:].isnan().all() and torch.equal(out[k][:first], clean[k][:first]), k
    for k in set(out) - {"dx", "dresidual", "dtoken_gate"}:
        assert out[k].isnan().all(), k
    mok.clear_status(ws)
    again = run()
    assert mok.read_status(ws) == 0 and all(torch.equal(again[k], clean[k]) for k in clean)
