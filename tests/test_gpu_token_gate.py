"""The gradient of the gate by token, against the plain 64-bit form, within the kernel's own roundings.

With u = 2^-24, g = dy weight and W = post gate the gradient is rho1 q, q = rho2 (s3 + c2 s4) + s5, c2 = - rho2^2 s1
/ d, of four sums of d products: s1 of h g, s3 of g W x, s4 of h W x, s5 of dres W x.  A product has up to three
roundings before it is added, a sum at most d / 1024 + 40 additions (a thread's vectors, a warp's lanes, the
warps), a root half of its sum's error: with K = d / 1024 + 52, which leaves some for the last few operations,
s_i is off by at most K u of the sum of its terms' magnitudes, m_i, and rho by K / 2 u of itself.  So q is off by at
most K u (rho2 (2 m3 + 4 rho2^2 m1 m4 / d) + 2 m5), the factors counting rho2 and rho1, c2's three and s4."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_14_gb300 as mok
from tests import _around, _block
from tests._helpers import ensure_lib, f64

pytestmark = pytest.mark.gpu


def _packed(t):
    """Codes and scales of a tensor by the 64-bit rule, and the values that they hold."""
    a = f64(t)
    s, _ = _around.mx_exponents(a)
    q = torch.from_numpy(a / np.repeat(2.0 ** s, 32, axis=-1)).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    return ((q.view(torch.uint8).cuda(), torch.from_numpy((s + 127).astype(np.uint8)).cuda()),
            q.double().numpy() * np.repeat(2.0 ** s, 32, axis=-1))


@pytest.mark.parametrize("T,d,res,packed", [
    (40, 64, "bf16", False), (700, 512, "f32", False), (517, 1544, "f32", False), (330, 4096, "bf16", True),
    (330, 7168, "bf16", False), (330, 7168, "f32", True), (170, 8192, "bf16", True), (40, 12288, "bf16", False),
    (40, 32768, "f32", False)])
@pytest.mark.parametrize("next_norm,dh", [(True, True), (True, False), (False, True)])
def test_token_gate(T, d, res, packed, next_norm, dh):
    ensure_lib()
    g = torch.Generator().manual_seed(T + d)
    rt = torch.float32 if res == "f32" else torch.bfloat16
    x, h = torch.randn((T, d), generator=g).bfloat16(), torch.randn((T, d), generator=g) * torch.exp(0.5 * torch.randn((T, 1), generator=g))
    h[:, ::max(1, d // 5)] *= 20.0
    h = h.to(rt)
    post, weight, gate = (1 + 0.1 * torch.randn(d, generator=g) for _ in range(3))
    tg = torch.rand(T, generator=g)
    dy = (0.01 * torch.randn((T, d), generator=g)).bfloat16() if next_norm else None
    dres = (0.01 * torch.randn((T, d), generator=g)).to(rt) if dh else None
    nx, nh, dev_x, dev_h = f64(x), f64(h), x.cuda(), h.cuda()
    if packed:
        (dev_x, nx), (dev_h, nh) = _packed(x), _packed(h)
    put = lambda t: None if t is None else t.cuda()  # noqa: E731
    out = mok.sandwich_norm_backward(dev_x, dev_h if next_norm else None, put(post), dy=put(dy), dres=put(dres),
                                     weight=put(weight) if next_norm else None, gate=put(gate), token_gate=put(tg),
                                     residual_dtype=rt)
    n = lambda t: None if t is None else f64(t)  # noqa: E731
    kw = dict(weight=n(weight)) if next_norm else {}
    ref = _block.sandwich_grad(nx, nh, n(post), n(dy), n(dres), gate=n(gate), token_gate=n(tg), **kw)["dtoken_gate"]
    rho = lambda v: 1.0 / np.sqrt((v * v).mean(1) + 1e-6)  # noqa: E731
    wx = np.abs(n(post) * n(gate) * nx)
    m = 0.0 if dres is None else 2 * (np.abs(n(dres)) * wx).sum(1)
    if next_norm:
        gg, r2 = np.abs(n(dy) * n(weight)), rho(nh)
        m = m + r2 * (2 * (gg * wx).sum(1) + 4 * r2 ** 2 * (np.abs(nh) * gg).sum(1) * (np.abs(nh) * wx).sum(1) / d)
    tol = (d / 1024 + 52) * 2.0 ** -24 * rho(nx) * m
    assert (np.abs(f64(out["dtoken_gate"]) - ref) <= tol).all()
    # What the tolerance is worth, by the plain form alone: at 32768 terms it is 0.4% of a gradient in the
    # median, so that a factor wrong by one part in a hundred shows in 80% of the rows, more where d is less.
    assert (0.01 * np.abs(ref) > tol).mean() > 0.75
