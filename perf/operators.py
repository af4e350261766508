"""The operators around the expert layer in a training or serving step, as cases that can be timed.

Five operators: the RMS norm in front of the layer (with the residual's addition and an optional
MXFP8 output) and its backward pass, the router's balance and z losses with per-expert counts and
the logits' gradient, the norm of all gradients with its clipping factor, and AdamW over all
weights at once with states in 32 or in 8 bits.  Each has a plain form in elementary torch
operations (fp32 arithmetic, one rounding at the end), the library's call, and a definition in
64 bits.

Sizes are those of the layer workloads (d = 7168, F = 2048, E = 256 or 384, k = 8; the tiny layer
with d = 256, E = 8, k = 2, F = 128) and odd ones of the same range.
"""

import math

import torch

own = False

EPS = 1e-6
BETAS, ADAM_EPS, LR, DECAY, STEP = (0.9, 0.95), 1e-8, 3e-4, 0.1, 100
MAX_NORM = 1.0
ALPHA = 1e-2
FLOATS = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token of a decoding sequence: nothing but latency
        dict(name="norm_one_token", op="norm", T=1, d=7168, residual="bf16", weight="bf16", mx=False),
        # an odd number of tokens, width no multiple of 128, a residual stream kept in fp32
        dict(name="norm_odd_f32", op="norm", T=2999, d=2056, residual="f32", weight="f32", mx=False),
        # the MXFP8 layer's whole batch: bf16 rows for the router, codes and scales for the experts
        dict(name="norm_prompt_mx", op="norm", T=16384, d=7168, residual="bf16", weight="bf16", mx=True),
        # backward of a small odd micro-batch, the residual stream's gradient in fp32
        dict(name="norm_grad_odd_f32", op="norm_grad", T=517, d=1544, residual="f32", weight="f32"),
        # backward at the training workload's batch
        dict(name="norm_grad_train", op="norm_grad", T=8192, d=7168, residual="bf16", weight="bf16"),
        # the tiny layer's batch, one sequence
        dict(name="balance_tiny", op="balance", T=256, E=8, k=2, S=1, masked=False, z=0.0),
        # a packed batch of ragged sequences with padding tokens, balanced per sequence, with z loss
        dict(name="balance_packed", op="balance", T=16384, E=384, k=8, S=37, masked=True, z=1e-3),
        # the gradients of twelve tiny layers (96 tensors)
        dict(name="grad_norm_tiny", op="grad_norm", L=12, E=8, d=256, F=128),
        # the gradients of 32 experts at full width
        dict(name="grad_norm_experts", op="grad_norm", L=1, E=32, d=7168, F=2048),
        # twelve tiny layers, 96 tensors, fp32 states
        dict(name="adamw_tiny", op="adamw", L=12, E=8, d=256, F=128, states="f32"),
        # 32 experts at full width, fp32 states
        dict(name="adamw_experts", op="adamw", L=1, E=32, d=7168, F=2048, states="f32"),
        # the same with states in 8 bits
        dict(name="adamw_experts_mx", op="adamw", L=1, E=32, d=7168, F=2048, states="mxfp8"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm_grad", "balance", "grad_norm", "adamw"])
    if op == "norm":
        mx = rng.random() < 0.5
        d = 128 * log(1, 56) if mx else 8 * log(8, 896)
        return dict(op=op, T=log(1, 16384), d=d, residual=rng.choice(["none", "bf16", "f32"]),
                    weight=rng.choice(["bf16", "f32"]), mx=mx)
    if op == "norm_grad":
        return dict(op=op, T=log(1, 8192), d=8 * log(8, 896), residual=rng.choice(["none", "bf16", "f32"]),
                    weight=rng.choice(["bf16", "f32"]))
    if op == "balance":
        E = 8 * log(1, 48)
        return dict(op=op, T=log(1, 16384), E=E, k=rng.randint(1, 8), S=log(1, 64),
                    masked=rng.random() < 0.5, z=rng.choice([0.0, 1e-3]))
    c = dict(op=op, L=log(1, 12), E=log(1, 32), d=log(48, 7168), F=log(32, 2048))
    while c["L"] * (c["E"] + 1) * c["d"] * c["F"] > 4.8e8:
        c["L"], c["E"] = max(1, c["L"] // 2), max(1, (c["E"] * 2) // 3)
    if op == "adamw":
        c["states"] = rng.choice(["f32", "mxfp8"])
    return c


# ------------------------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _hidden(g, T, d, dtype):
    """Rows of a residual stream: normal, every row with its own size and a few large channels."""
    v = torch.randn((T, d), generator=g, device="cuda")
    v *= torch.exp(0.5 * torch.randn((T, 1), generator=g, device="cuda"))
    v[:, ::max(1, d // 5)] *= 20.0
    return v.to(dtype)


def _sizes(case):
    """Element counts of L layers' weights: (bf16 tensors, fp32 tensors)."""
    L, E, d, F = case["L"], case["E"], case["d"], case["F"]
    return [d * E, E * d * F, E * d * F, E * F * d, d * F, d * F, F * d] * L, [d] * L


def _spans(sizes):
    """Places of the tensors in one flat buffer, each start at a multiple of 32 elements."""
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += (n + 31) // 32 * 32
    return starts, at


def _parts(flat, sizes):
    starts, _ = _spans(sizes)
    return [flat[s:s + n] for s, n in zip(starts, sizes)]


def _flat(g, sizes, std, dtype):
    """A flat buffer of normal values with zeros between the tensors."""
    starts, total = _spans(sizes)
    v = _normal(g, (total,), std, dtype)
    for s, n in zip(starts, sizes):
        v[s + n:(s + n + 31) // 32 * 32] = 0
    return v


def _group(g, sizes, low, states):
    """One group of weights with gradients and optimiser states, each in a flat buffer."""
    w = _flat(g, sizes, 0.02, torch.float32)
    gr = {"grad": _flat(g, sizes, 1e-3, torch.bfloat16 if low else torch.float32)}
    m = _flat(g, sizes, 3e-4, torch.float32)
    v = _flat(g, sizes, 1e-3, torch.float32).square_()
    if low:
        gr["param"], gr["master"] = w.to(torch.bfloat16), w
    else:
        gr["param"] = w
    if states == "mxfp8":
        for key, x in (("m", m), ("v", v)):
            codes, scales = _mx(x.view(-1, 32))
            gr[key], gr[key + "_scale"] = codes.view(-1), scales.view(-1)
        starts, total = _spans(sizes)
        place = torch.arange(total, device="cuda")
        for s, n in zip(starts, sizes):
            place[s:(s + n + 31) // 32 * 32] -= s
        gr["place"] = place.to(torch.int32)  # every element's index in its own tensor
    else:
        gr["m"], gr["v"] = m, v
    return gr


def _adam_handle(st):
    """What a user's program keeps: the optimiser over the weights, and the list of gradients."""
    import mixture_experts_layer_14_gb300 as mok

    params, grads, decay = [], [], []
    state = {key: [] for key in ("master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")}
    for key, wd in (("low", DECAY), ("full", 0.0)):
        gr, sizes = st[key], st[key + "_sizes"]
        params += _parts(gr["param"], sizes)
        grads += _parts(gr["grad"], sizes)
        decay += [wd] * len(sizes)
        state["master"] += _parts(gr["master"], sizes) if "master" in gr else [None] * len(sizes)
        for short, name in (("m", "exp_avg"), ("v", "exp_avg_sq")):
            if st["states"] == "mxfp8":
                state[name] += [c.view(torch.uint8) for c in _parts(gr[short], sizes)]
                sc = gr[short + "_scale"].view(torch.uint8)
                state[name + "_scale"] += [
                    sc[s // 32:s // 32 + (n + 31) // 32] for s, n in zip(_spans(sizes)[0], sizes)]
            else:
                state[name] += _parts(gr[short], sizes)
    opt = mok.AdamW(params, betas=BETAS, eps=ADAM_EPS, weight_decay=decay, states=st["states"],
                    state=state, step=STEP)
    return opt, mok.TensorList(grads)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        st["x"] = _normal(g, (T, d), 1.0, torch.bfloat16)
        st["r"] = None if case["residual"] == "none" else _hidden(g, T, d, FLOATS[case["residual"]])
        st["w"] = (1.0 + 0.1 * torch.randn((d,), generator=g, device="cuda")).to(FLOATS[case["weight"]])
    elif case["op"] == "norm_grad":
        T, d = case["T"], case["d"]
        kind = torch.float32 if case["residual"] == "f32" else torch.bfloat16
        st["s"] = _hidden(g, T, d, kind)
        st["dy"] = _normal(g, (T, d), 1e-2, torch.bfloat16)
        st["dres"] = None if case["residual"] == "none" else _normal(g, (T, d), 1e-2, kind)
        st["w"] = (1.0 + 0.1 * torch.randn((d,), generator=g, device="cuda")).to(FLOATS[case["weight"]])
        st["ws"] = None
        if own:  # a training program keeps the workspace
            import mixture_experts_layer_14_gb300 as mok

            st["ws"] = torch.zeros(mok.rms_norm_workspace_size(T, d), dtype=torch.uint8, device="cuda")
    elif case["op"] == "balance":
        T, E, S, k = case["T"], case["E"], case["S"], min(case["k"], case["E"])
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1.0
        st["logits"] = _normal(g, (T, E)) - 0.5 * torch.log(rank)  # some experts are liked more
        st["idx"] = st["logits"].topk(k, dim=1).indices.to(torch.int32)
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
        ends = torch.tensor([0, T], device="cuda")
        st["offsets"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32) if S > 1 else None
        st["mask"] = (torch.rand((T,), generator=g, device="cuda") < 0.9) if case["masked"] else None
        if own:  # a training program keeps the workspace and the layer's sizes
            import mixture_experts_layer_14_gb300 as mok

            st["D"] = mok.dims(T, 128, E, k, 128, 0, 0)
            st["ws"] = torch.zeros(mok.balance_loss_workspace_size(st["D"], S), dtype=torch.uint8,
                                   device="cuda")
    elif case["op"] == "grad_norm":
        low, full = _sizes(case)
        st["low"], st["full"] = _flat(g, low, 1e-3, torch.bfloat16), _flat(g, full, 1e-3, torch.float32)
        if own:  # a training program keeps the list of its gradient buffers and the workspace
            import mixture_experts_layer_14_gb300 as mok

            st["grads"] = mok.TensorList(_parts(st["low"], low) + _parts(st["full"], full))
            st["ws"] = torch.zeros(mok.grad_norm_workspace_size(st["grads"]), dtype=torch.uint8,
                                   device="cuda")
    else:
        st["low_sizes"], st["full_sizes"] = _sizes(case)
        st["low"] = _group(g, st["low_sizes"], True, case["states"])
        st["full"] = _group(g, st["full_sizes"], False, case["states"])
        st["clip"] = torch.tensor([2.0, 0.5], device="cuda")  # {norm, factor} as grad_norm gives it
        st["step"] = STEP
        if own:
            st["opt"], st["grads"] = _adam_handle(st)
    return st


# ------------------------------------------------------------------------------- the plain forms
def _mx(v):
    """E4M3 codes and power-of-two scales of blocks of 32 along the last dimension: the scale is
    2^s with s the smallest integer such that the block's largest magnitude is <= 448 * 2^s."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    scale, inverse = _mx_scale(b)
    q = (b * inverse.unsqueeze(-1)).clamp_(-448.0, 448.0)
    return q.to(torch.float8_e4m3fn).view(v.shape), scale


def _mx_scale(b):
    """Each block's scale 2^s and 2^-s, both exact."""
    mant, e = torch.frexp(b.abs().amax(-1))
    s = torch.where(mant == 0, -127, e - 9 + (mant > 0.875).to(e.dtype)).clamp_(-127, 127)
    return (s + 127).to(torch.uint8).view(torch.float8_e8m0fnu), ((127 - s) << 23).view(torch.float32)


def _norm(st):
    h = st["x"].float()
    if st["r"] is not None:
        h = h + st["r"].float()
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    v = h * rstd * st["w"].float()
    out = {"y": v.to(torch.bfloat16)}
    if st["r"] is not None:
        out["residual"] = h.to(st["r"].dtype)
    if st["mx"]:
        out["codes"], out["scales"] = _mx(v)
    return out


def _norm_grad(st):
    s, dy, w = st["s"].float(), st["dy"].float(), st["w"].float()
    rstd = torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS)
    xhat = s * rstd
    gy = dy * w
    ds = rstd * (gy - xhat * (gy * xhat).mean(-1, keepdim=True))
    if st["dres"] is not None:
        ds = ds + st["dres"].float()
    out = {"dx": ds.to(torch.bfloat16), "dweight": (dy * xhat).sum(0)}
    if st["residual"] == "f32":
        out["dresidual"] = ds
    return out


def _balance(st):
    logits, idx = st["logits"], st["idx"].long()
    (T, E), k, S, dev = logits.shape, idx.shape[1], st["S"], logits.device
    valid = torch.ones(T, device=dev) if st["mask"] is None else st["mask"].float()
    seq = torch.zeros(T, dtype=torch.long, device=dev)
    if st["offsets"] is not None:
        seq = (torch.arange(T, device=dev).unsqueeze(1) >= st["offsets"][1:-1].unsqueeze(0)).sum(1)
    counts = torch.zeros(S * E, dtype=torch.int32, device=dev)
    counts.index_add_(0, (seq.unsqueeze(1) * E + idx).reshape(-1),
                      valid.to(torch.int32).unsqueeze(1).expand(T, k).reshape(-1))
    counts = counts.view(S, E)
    n_seq = torch.zeros(S, device=dev).index_add_(0, seq, valid)
    n = n_seq.sum().clamp(min=1.0)
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    p, lse = e / total, (top + torch.log(total)).squeeze(1)
    c = counts[seq].float()
    inner = (c * p).sum(1)
    a = valid * (ALPHA * E / k) / (n * n_seq[seq].clamp(min=1.0))
    b = valid * (2.0 * st["z"]) / n
    loss = torch.stack([(a * inner).sum(), 0.5 * (b * lse * lse).sum()])
    dlogits = p * (a.unsqueeze(1) * (c - inner.unsqueeze(1)) + (b * lse).unsqueeze(1))
    return {"loss": loss, "counts": counts, "dlogits": dlogits}


def _grad_norm(st):
    n = torch.sqrt(st["low"].float().square_().sum() + st["full"].square().sum())
    return torch.stack([n, torch.clamp(MAX_NORM / n, max=1.0)])


def _dither(place, step):
    """16 + 16 bits for every element and step, in [0, 2^16): thresholds of m and of v."""
    x = (place.long() * 0x85EBCA6B + step * 0x9E3779B9) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x2C1B3C6D) & 0xFFFFFFFF
    x = ((x ^ (x >> 12)) * 0x297A2D39) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    return (x >> 16).to(torch.int32), (x & 0xFFFF).to(torch.int32)


def _mx_dither(x, r, never_zero):
    """Codes and scales of x, rounded up where the element's threshold says so."""
    b = x.view(-1, 32)
    scale, inverse = _mx_scale(b)
    q = (b.abs() * inverse.unsqueeze(-1)).view(-1)
    bits = (q.view(torch.int32) + (r << 4) + 8) & ~0xFFFFF                   # 3 bits of mantissa
    small = torch.floor(q * 512.0 + (r.float() + 0.5) * 2.0 ** -16) * 2.0 ** -9  # multiples of 2^-9
    q = torch.where(q < 2.0 ** -6, small, bits.view(torch.float32)).clamp_(max=448.0)
    if never_zero:
        q = torch.where(x > 0, q.clamp(min=2.0 ** -9), q)
    return torch.copysign(q, x).to(torch.float8_e4m3fn), scale


def _unpack(codes, scales):
    return (codes.float().view(-1, 32) * scales.float().unsqueeze(1)).view(-1)


def _adam_group(gr, step, clip, decay, mx):
    g = gr["grad"].float() * clip
    m = _unpack(gr["m"], gr["m_scale"]) if mx else gr["m"]
    v = _unpack(gr["v"], gr["v_scale"]) if mx else gr["v"]
    w = gr["master"] if "master" in gr else gr["param"]
    m.mul_(BETAS[0]).add_(g * (1.0 - BETAS[0]))
    v.mul_(BETAS[1]).add_(g.square_().mul_(1.0 - BETAS[1]))
    root = torch.sqrt(v * (1.0 / (1.0 - BETAS[1] ** step))).add_(ADAM_EPS)
    w.sub_((m * (1.0 / (1.0 - BETAS[0] ** step))).div_(root).add_(w * decay).mul_(LR))
    if "master" in gr:
        gr["param"].copy_(w)
    if mx:
        rm, rv = _dither(gr["place"], step)
        codes, scales = _mx_dither(m, rm, False)
        gr["m"].copy_(codes), gr["m_scale"].copy_(scales)
        codes, scales = _mx_dither(v, rv, True)
        gr["v"].copy_(codes), gr["v_scale"].copy_(scales)


def _adam_outputs(st):
    return {key: {k: v for k, v in st[key].items() if k not in ("grad", "place")} for key in ("low", "full")}


def _adamw(st):
    st["step"] += 1
    _adam_group(st["low"], st["step"], st["clip"][1], DECAY, st["states"] == "mxfp8")
    _adam_group(st["full"], st["step"], st["clip"][1], 0.0, st["states"] == "mxfp8")
    return _adam_outputs(st)


PLAIN = {"norm": _norm, "norm_grad": _norm_grad, "balance": _balance, "grad_norm": _grad_norm, "adamw": _adamw}


# ------------------------------------------------------------------------------- one pass
def run(st):
    if not own:
        return PLAIN[st["op"]](st)
    import mixture_experts_layer_14_gb300 as mok

    if st["op"] == "norm":
        o = mok.rms_norm(st["x"], st["w"], EPS, residual=st["r"], mx="rows" if st["mx"] else None)
        if st["mx"]:
            o["codes"], o["scales"] = o["codes"].view(torch.float8_e4m3fn), o["scales"].view(torch.float8_e8m0fnu)
        return o
    if st["op"] == "norm_grad":
        return mok.rms_norm_backward(st["dy"], st["s"], st["w"], EPS, dres=st["dres"], ws=st["ws"])
    if st["op"] == "balance":
        return mok.balance_loss(st["D"], st["logits"], st["idx"], st["ws"], ALPHA, z_coef=st["z"],
                                seq_offsets=st["offsets"], token_mask=st["mask"])
    if st["op"] == "grad_norm":
        return mok.grad_norm(st["grads"], MAX_NORM, ws=st["ws"])
    st["opt"].step(st["grads"], LR, clip=st["clip"])
    return _adam_outputs(st)


# ------------------------------------------------------------------------------- the work of one pass
def work(case):
    if case["op"] in ("norm", "norm_grad"):
        n, d = case["T"] * case["d"], case["d"]
        res = {"none": 0, "bf16": 2, "f32": 4}[case["residual"]]
        w = 2 if case["weight"] == "bf16" else 4
        if case["op"] == "norm":
            return {"bytes": n * (2 + 2 * res + 2 + (33 / 32 if case["mx"] else 0)) + w * d, "flops": 5 * n}
        s = max(res, 2)
        return {"bytes": n * (2 + s + res + 2 + (4 if case["residual"] == "f32" else 0)) + (w + 4) * d,
                "flops": 11 * n}
    if case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], min(case["k"], case["E"]), case["S"]
        return {"bytes": 8 * T * E + 4 * T * k + (T if case["masked"] else 0) + 4 * S * E + 4 * (S + 1) + 8,
                "flops": 11 * T * E}
    low, full = _sizes(case)
    low, full = sum(low), sum(full)
    if case["op"] == "grad_norm":
        return {"bytes": 2 * low + 4 * full + 8, "flops": 2 * (low + full)}
    state = 16 if case["states"] == "f32" else 4 * 33 / 32  # m and v, read and written
    return {"bytes": low * (2 + 2 + 8 + state) + full * (4 + 8 + state), "flops": 16 * (low + full)}


# ------------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "norm":
        h = st["x"].to(f8)
        h = h if st["r"] is None else h.add_(st["r"])
        power = torch.linalg.vector_norm(h, dim=1).square() / case["d"]
        out = {"residual": None if st["r"] is None else h.clone()}
        h /= (power + EPS).sqrt().unsqueeze(1)
        h *= st["w"]
        out["y"] = h
        if case["mx"]:  # codes: the unrounded quotient; scales: whole powers of two, no such value
            s = torch.ceil(torch.log2(h.view(-1, 32).abs().amax(1) / 448.0)).clamp(-127, 127)
            out["codes"] = (h.view(-1, 32) * torch.exp2(-s).unsqueeze(1)).view(h.shape)
            out["scales"] = None
        return {k: v for k, v in out.items() if v is not None or k == "scales"}
    if case["op"] == "norm_grad":
        s, gy = st["s"].to(f8), st["dy"].to(f8) * st["w"].to(f8)
        var = torch.einsum("td,td->t", s, s) / case["d"] + EPS
        dot = torch.einsum("td,td->t", s, gy) / case["d"]
        dw = torch.einsum("td,td,t->d", s, st["dy"].to(f8), var ** -0.5)
        ds = gy * (var ** -0.5).unsqueeze(1) - s * (dot * var ** -1.5).unsqueeze(1)
        if st["dres"] is not None:
            ds += st["dres"]
        out = {"dx": ds, "dweight": dw}
        return dict(out, dresidual=ds) if case["residual"] == "f32" else out
    if case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], st["idx"].shape[1], case["S"]
        bounds = [0, T] if st["offsets"] is None else st["offsets"].tolist()
        alive = torch.ones(T, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"]
        n = max(1, int(alive.sum()))
        lg = st["logits"].to(f8)
        lse = torch.logsumexp(lg, 1)
        p = torch.exp(lg - lse.unsqueeze(1))
        chosen = torch.zeros((T, E), dtype=f8, device="cuda").scatter_(1, st["idx"].long(), 1.0)
        dl, balance = torch.zeros_like(lg), 0.0
        for a, b in zip(bounds[:-1], bounds[1:]):
            ok = alive[a:b].to(f8)
            m = float(ok.sum())
            if m == 0:
                continue
            load, mean = ok @ chosen[a:b], ok @ p[a:b] / m
            f = load * (E / (k * m))
            balance += ALPHA * m / n * float(f @ mean)
            q = p[a:b]
            dl[a:b] = (ALPHA / n) * ok.unsqueeze(1) * q * (f - (q @ f).unsqueeze(1))
        ok = alive.to(f8)
        z = case["z"] / n * float((ok * lse * lse).sum())
        dl += (2.0 * case["z"] / n) * (ok * lse).unsqueeze(1) * p
        return {"loss": torch.tensor([balance, z], dtype=f8), "counts": None, "dlogits": dl}
    if case["op"] == "grad_norm":
        square = 0.0
        for flat in (st["low"], st["full"]):
            for at in range(0, flat.numel(), 1 << 28):
                part = flat[at:at + (1 << 28)].to(f8)
                square += float(part @ part)
        n = math.sqrt(square)
        return torch.tensor([n, min(1.0, MAX_NORM / n)], dtype=f8)
    out, t = {}, STEP + 1
    for key, decay in (("low", DECAY), ("full", 0.0)):
        gr = st[key]
        g = gr["grad"].to(f8) * 0.5
        if case["states"] == "mxfp8":
            wide = lambda k: (gr[k].to(f8).view(-1, 32) * gr[k + "_scale"].to(f8).unsqueeze(1)).view(-1)  # noqa: E731
            m, v = wide("m"), wide("v")
        else:
            m, v = gr["m"].to(f8), gr["v"].to(f8)
        w = gr["master" if key == "low" else "param"].to(f8)
        m = BETAS[0] * m + (1.0 - BETAS[0]) * g
        v = BETAS[1] * v + (1.0 - BETAS[1]) * g * g
        del g
        w = w - LR * ((m / (1.0 - BETAS[0] ** t)) / ((v / (1.0 - BETAS[1] ** t)).sqrt() + ADAM_EPS) + decay * w)
        res = {"param": w}
        if key == "low":
            res["master"] = w
        for name, x in (("m", m), ("v", v)):
            if case["states"] == "mxfp8":  # the unrounded quotient in place of the codes
                b = x.view(-1, 32)
                s = torch.ceil(torch.log2(b.abs().amax(1) / 448.0)).clamp(-127, 127)
                res[name], res[name + "_scale"] = (b * torch.exp2(-s).unsqueeze(1)).view(-1), None
            else:
                res[name] = x
        out[key] = res
    return out
