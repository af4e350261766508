"""The operators of a block with grouped routing, norms on both sides and 8-bit checkpoints, as
cases that can be timed.

Six operators: the choice of experts from router logits (softmax or sigmoid scores, a bias that only
ranks, groups, top-k, renormalised weights) and its backward pass; the norm after a branch fused
with its gate, the scaled residual and the next norm (optionally with MXFP8 output and an 8-bit
checkpoint of what the backward pass reads) and its backward pass, from the tensors or from their
8-bit form; and activations into 8 bits and back.  Each has a plain form in elementary torch
operations, the library's call, and a definition in 64 bits.

Sizes are those of the layer workloads (d = 7168, F = 2048, E = 256 or 384, k = 8, T to 16384) and
odd ones of the same range.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-6
RES_SCALE = 0.75  # the residual's factor in the norm's cases
FLOATS = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a decoding step of 64 sequences: sigmoid scores, balance bias, 4 of 8 groups by their top two
        dict(name="select_decode", op="select", T=64, E=256, k=8, scoring="sigmoid", bias=True, groups=8, kept=4,
             by="top2", renorm=True, scale=2.5, masked=False),
        # the whole batch of the layer with 384 experts: sigmoid scores and bias, no groups
        dict(name="select_prompt", op="select", T=16384, E=384, k=8, scoring="sigmoid", bias=True, groups=1, kept=1,
             by="max", renorm=True, scale=2.827, masked=False),
        # an odd micro-batch, softmax scores that are not renormalised (the gradient is dense)
        dict(name="select_grad_odd", op="select_grad", T=517, E=160, k=6, scoring="softmax", renorm=False,
             scale=16.0, aux=False, masked=False),
        # the training batch: sigmoid scores, the gradient of the balance loss joins in
        dict(name="select_grad_train", op="select_grad", T=8192, E=256, k=8, scoring="sigmoid", renorm=True,
             scale=2.5, aux=True, masked=False),
        # one token of a decoding sequence: nothing but latency
        dict(name="sandwich_one_token", op="sandwich", T=1, d=7168, residual="bf16", weight="bf16", gate="none",
             next=True, mx=False, save=False),
        # the training batch of an MXFP8 layer: codes for the experts, and what the backward pass needs in 8 bits
        dict(name="sandwich_prompt_save", op="sandwich", T=16384, d=7168, residual="bf16", weight="bf16",
             gate="channel", next=True, mx=True, save=True),
        # an odd micro-batch of an fp32 residual stream, width no multiple of 128, gates by token and by channel
        dict(name="sandwich_grad_odd_f32", op="sandwich_grad", T=517, d=1544, residual="f32", weight="f32",
             gate="both", next=True, dh=True, packed=False),
        # the training batch, from the 8-bit checkpoint
        dict(name="sandwich_grad_train", op="sandwich_grad", T=8192, d=7168, residual="bf16", weight="bf16",
             gate="channel", next=True, dh=True, packed=True),
        # gate activations of a decode-sized micro-batch in fp32, as the MXFP8 layer saves them
        dict(name="pack_small_f32", op="pack", rows=512, K=2048, type="f32"),
        # gate activations of every route of the training batch
        dict(name="pack_routes", op="pack", rows=65536, K=2048, type="bf16"),
        # and back: an odd number of narrow rows
        dict(name="unpack_odd", op="unpack", rows=1999, K=256, type="bf16"),
        # back to fp32 for the MXFP8 layer's backward pass
        dict(name="unpack_routes_f32", op="unpack", rows=65536, K=2048, type="f32"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["select", "select_grad", "sandwich", "sandwich_grad", "pack", "unpack"])
    if op in ("select", "select_grad"):
        T, scoring, renorm = log(1, 16384), rng.choice(["softmax", "sigmoid"]), rng.random() < 0.7
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = groups * max(8 // min(groups, 8), 8 * log(1, 48) // groups)
        kept = groups if op == "select_grad" else rng.randint(1, groups)
        k = rng.randint(1, min(8, kept * (E // groups)))
        c = dict(op=op, T=T, E=E, k=k, scoring=scoring, renorm=renorm, scale=rng.choice([1.0, 2.5]),
                 masked=rng.random() < 0.3)
        if op == "select_grad":
            return dict(c, aux=rng.random() < 0.5)
        return dict(c, bias=rng.random() < 0.7, groups=groups, kept=kept, by=rng.choice(["max", "top2"]))
    if op in ("sandwich", "sandwich_grad"):
        eight = rng.random() < 0.5
        residual = rng.choice(["bf16", "f32"])
        c = dict(op=op, T=log(1, 16384 if op == "sandwich" and residual == "bf16" else 8192),
                 d=128 * log(1, 56) if eight else 8 * log(8, 896), residual=residual, weight=rng.choice(["bf16", "f32"]),
                 gate=rng.choice(["none", "channel", "token", "both"]), next=rng.random() < 0.8)
        if op == "sandwich":
            return dict(c, mx=eight and c["next"] and rng.random() < 0.7, save=eight and rng.random() < 0.7)
        return dict(c, dh=not c["next"] or rng.random() < 0.7, packed=eight)
    K = 32 * log(1, 64)
    return dict(op=op, rows=min(log(1, 65536), 134217728 // K), K=K, type=rng.choice(["bf16", "f32"]))


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


def _logits(g, T, E, masked):
    """Router logits; some experts are liked more.  Masked: a tenth of the experts is shut off, and
    every fiftieth token has none left."""
    rank = torch.randperm(E, generator=g, device="cuda").float() + 1.0
    l = _normal(g, (T, E)) - 0.5 * torch.log(rank)
    if masked:
        l.masked_fill_(torch.rand((T, E), generator=g, device="cuda") < 0.1, -math.inf)
        l[::50] = -math.inf
    return l


def _selection(case):
    """What a user's program keeps: the rule by which its router chooses, and a workspace."""
    import mixture_experts_layer_14_gb300 as mok

    D = mok.dims(case["T"], 128, case["E"], case["k"], 128, 0, 0)
    sel = mok.Selection(scoring=case["scoring"], n_groups=case.get("groups", 1), topk_groups=case.get("kept", 1),
                        group_score=case.get("by", "max"), renormalise=case["renorm"], scale=case["scale"])
    return D, sel, torch.zeros(mok.workspace_size(D), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] in ("select", "select_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = _logits(g, T, E, case["masked"])
        if case["op"] == "select":  # the balance bias moves in steps of 1e-3
            st["b"] = torch.randint(-50, 51, (E,), generator=g, device="cuda") * 1e-3 if case["bias"] else None
        else:
            st["idx"] = st["logits"].topk(k, dim=1).indices.to(torch.int32)
            st["dw"] = _normal(g, (T, k), 1e-2)
            st["daux"] = _normal(g, (T, E), 1e-4) if case["aux"] else None
        if own:
            st["D"], st["sel"], st["ws"] = _selection(case)
    elif case["op"] in ("sandwich", "sandwich_grad"):
        T, d, kind = case["T"], case["d"], FLOATS[case["residual"]]

        def weight(mean):
            return (mean + 0.1 * torch.randn((d,), generator=g, device="cuda")).to(FLOATS[case["weight"]])

        st["x"] = _normal(g, (T, d), 1.0, torch.bfloat16)
        st["post"], st["w"] = weight(1.0), weight(1.0) if case["next"] else None
        st["cg"] = weight(0.5) if case["gate"] in ("channel", "both") else None
        st["tg"] = torch.rand((T,), generator=g, device="cuda") if case["gate"] in ("token", "both") else None
        if case["op"] == "sandwich":
            st["r"] = _hidden(g, T, d, kind)
        else:
            st["h"] = _hidden(g, T, d, kind)
            st["dy"] = _normal(g, (T, d), 1e-2, torch.bfloat16) if case["next"] else None
            st["dres"] = _normal(g, (T, d), 1e-2, kind) if case["dh"] else None
            if case["packed"]:  # the forward pass left codes and scales of x and h
                st["x"], st["h"] = _mx(st["x"].float()), _mx(st["h"].float())
            if own:  # a training program keeps the workspace
                import mixture_experts_layer_14_gb300 as mok

                st["ws"] = torch.zeros(mok.sandwich_norm_workspace_size(T, d), dtype=torch.uint8, device="cuda")
                if case["packed"]:
                    st["x"], st["h"] = (tuple(u.view(torch.uint8) for u in st[key]) for key in ("x", "h"))
    else:
        v = _hidden(g, case["rows"], case["K"], FLOATS[case["type"]])
        if case["op"] == "pack":
            st["x"] = v
        else:
            st["codes"], st["scales"] = _mx(v.float())
            if own:
                st["codes"], st["scales"] = st["codes"].view(torch.uint8), st["scales"].view(torch.uint8)
    return st


# ------------------------------------------------------------------------------- the plain forms
def _mx(v):
    """E4M3 codes and power-of-two scales of blocks of 32 along the last dimension: the scale is
    2^s with s the smallest integer such that the block's largest magnitude is <= 448 * 2^s."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    mant, e = torch.frexp(b.abs().amax(-1))
    s = torch.where(mant == 0, -127, e - 9 + (mant > 0.875).to(e.dtype)).clamp_(-127, 127)
    inverse = ((127 - s) << 23).view(torch.float32)
    q = (b * inverse.unsqueeze(-1)).clamp_(-448.0, 448.0)
    return q.to(torch.float8_e4m3fn).view(v.shape), (s + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _wide(packed):
    """fp32 values of codes and scales."""
    codes, scales = packed
    b = codes.float().view(*scales.shape, 32) * scales.float().unsqueeze(-1)
    return b.view(codes.shape)


def _scores(l, scoring):
    """Scores in the logits' own width; experts at -inf have none."""
    if scoring == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
    return e / e.sum(1, keepdim=True).clamp(min=torch.finfo(l.dtype).tiny)


def _select(st):
    l = st["logits"].double()  # in 64 bits: which of two near scores is larger decides
    T, E = l.shape
    s = _scores(l, st["scoring"])
    out = l == -math.inf
    c = s if st["b"] is None else s + st["b"].double()
    rank = l if st["b"] is None else c  # the scores rise with the logits
    c = c.masked_fill(out, -math.inf)
    kept = torch.ones((T, E), dtype=torch.bool, device=l.device)
    if st["groups"] > 1:
        top = c.view(T, st["groups"], -1).sort(dim=2, descending=True).values[:, :, :2]
        score = top[:, :, 0]
        if st["by"] == "top2" and top.shape[2] > 1:
            score = score + torch.where(top[:, :, 1] == -math.inf, 0.0, top[:, :, 1])
        best = score.sort(dim=1, descending=True, stable=True).indices[:, :st["kept"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, best, True)
        kept = keep.unsqueeze(2).expand(T, st["groups"], E // st["groups"]).reshape(T, E)
    rank = torch.where(kept, torch.where(out, -1e300, rank), -math.inf)
    idx = rank.sort(dim=1, descending=True, stable=True).indices[:, :st["k"]]
    w = s.gather(1, idx)
    if st["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return {"idx": idx.to(torch.int32), "w": (w * st["scale"]).float()}


def _select_grad(st):
    l, idx, dw = st["logits"], st["idx"].long(), st["dw"]
    s = _scores(l, st["scoring"])
    sj = s.gather(1, idx)
    if st["renorm"]:
        p = sj / sj.sum(1, keepdim=True).clamp(min=1e-37)
        inner = (p * dw).sum(1, keepdim=True)
        dl = p * (dw - inner) * (1.0 if st["scoring"] == "softmax" else 1.0 - sj)
        out = torch.zeros_like(l).scatter_(1, idx, dl * st["scale"])
    elif st["scoring"] == "sigmoid":
        out = torch.zeros_like(l).scatter_(1, idx, sj * (1.0 - sj) * dw * st["scale"])
    else:
        out = s * (torch.zeros_like(l).scatter_(1, idx, dw) - (sj * dw).sum(1, keepdim=True)) * st["scale"]
    return out if st["daux"] is None else out + st["daux"]


def _unit(v):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _sandwich(st):
    x = st["x"].float()
    n = _unit(x) * st["post"].float()
    if st["cg"] is not None:
        n = n * st["cg"].float()
    if st["tg"] is not None:
        n = n * st["tg"].unsqueeze(1)
    h = RES_SCALE * st["r"].float() + n
    out = {"residual": h.to(st["r"].dtype)}
    if st["next"]:
        v = _unit(h) * st["w"].float()
        out["y"] = v.to(torch.bfloat16)
        if st["mx"]:
            out["codes"], out["scales"] = _mx(v)
    if st["save"]:
        out["x_codes"], out["x_scales"] = _mx(x)
        out["h_codes"], out["h_scales"] = _mx(h)
    return out


def _sandwich_grad(st):
    x, h = (_wide(st[key]) if st["packed"] else st[key].float() for key in ("x", "h"))
    out = {}
    ds = 0.0 if st["dres"] is None else st["dres"].float()
    if st["next"]:
        dy = st["dy"].float()
        rho = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
        hhat, g = h * rho, dy * st["w"].float()
        ds = rho * (g - hhat * (g * hhat).mean(-1, keepdim=True)) + ds
        out["dweight"] = (dy * hhat).sum(0)
    post = st["post"].float()
    W = post if st["cg"] is None else post * st["cg"].float()
    rho = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xhat, gw = x * rho, ds * W
    q = (gw * xhat).sum(-1, keepdim=True)
    t = 1.0 if st["tg"] is None else st["tg"].unsqueeze(1)
    a = (ds * xhat * t).sum(0)
    out["dx"] = (rho * t * (gw - xhat * (q / st["d"]))).to(torch.bfloat16)
    out["dresidual"] = (RES_SCALE * ds).to(FLOATS[st["residual"]])
    out["dpost_weight"] = a if st["cg"] is None else a * st["cg"].float()
    if st["cg"] is not None:
        out["dgate"] = a * post
    if st["tg"] is not None:
        out["dtoken_gate"] = q.squeeze(1)
    return out


def _pack(st):
    codes, scales = _mx(st["x"].float())
    return {"codes": codes, "scales": scales}


def _unpack(st):
    return _wide((st["codes"], st["scales"])).to(FLOATS[st["type"]])


PLAIN = {"select": _select, "select_grad": _select_grad, "sandwich": _sandwich, "sandwich_grad": _sandwich_grad,
         "pack": _pack, "unpack": _unpack}


# ------------------------------------------------------------------------------- one pass
def _typed(out):
    """8-bit buffers as the numbers that they hold."""
    kinds = {"codes": torch.float8_e4m3fn, "scales": torch.float8_e8m0fnu}
    return {k: v.view(kinds[k.split("_")[-1]]) if k.split("_")[-1] in kinds else v for k, v in out.items()}


def run(st):
    if not own:
        return PLAIN[st["op"]](st)
    import mixture_experts_layer_14_gb300 as mok

    if st["op"] == "select":
        idx, w = mok.select_experts(st["D"], st["sel"], st["logits"], st["ws"], bias=st["b"])
        return {"idx": idx, "w": w}
    if st["op"] == "select_grad":
        return mok.select_experts_backward(st["D"], st["sel"], st["logits"], st["idx"], st["dw"], st["ws"],
                                           dlogits_aux=st["daux"])
    if st["op"] == "sandwich":
        return _typed(mok.sandwich_norm(
            st["x"], st["r"], st["post"], weight=st["w"], gate=st["cg"], token_gate=st["tg"], res_scale=RES_SCALE,
            eps=EPS, mx="rows" if st["mx"] else None, save="mxfp8" if st["save"] else None))
    if st["op"] == "sandwich_grad":
        return mok.sandwich_norm_backward(
            st["x"], st["h"], st["post"], dy=st["dy"], dres=st["dres"], weight=st["w"], gate=st["cg"],
            token_gate=st["tg"], res_scale=RES_SCALE, eps=EPS, residual_dtype=FLOATS[st["residual"]], ws=st["ws"])
    if st["op"] == "pack":
        codes, scales = mok.activation_pack(st["x"])
        return _typed({"codes": codes, "scales": scales})
    return mok.activation_unpack(st["codes"], st["scales"], FLOATS[st["type"]])


# ------------------------------------------------------------------------------- the work of one pass
def work(case):
    if case["op"] == "select":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 8 * T * E}
    if case["op"] == "select_grad":
        T, E, k = case["T"], case["E"], case["k"]
        dense = case["scoring"] == "softmax" and not case["renorm"]
        return {"bytes": 4 * T * E * (1 + case["aux"] + dense) + 8 * T * k + (0 if dense else 4 * T * k),
                "flops": T * E * (1 + 6 * dense) + 8 * T * k}
    if case["op"] in ("sandwich", "sandwich_grad"):
        T, d = case["T"], case["d"]
        n, r, w = T * d, 2 if case["residual"] == "bf16" else 4, 2 if case["weight"] == "bf16" else 4
        vectors = 1 + case["next"] + (case["gate"] in ("channel", "both"))
        tokens = 4 * T if case["gate"] in ("token", "both") else 0
        if case["op"] == "sandwich":
            per = 2 + 2 * r + 2 * case["next"] + 33 / 32 * (case["mx"] + 2 * case["save"])
            return {"bytes": n * per + vectors * w * d + tokens, "flops": 12 * n}
        saved = 33 / 32 * (1 + case["next"]) if case["packed"] else 2 + r * case["next"]
        per = saved + 2 * case["next"] + r * case["dh"] + 2 + r
        return {"bytes": n * per + vectors * (w + 4) * d + 2 * tokens, "flops": 24 * n}
    n = case["rows"] * case["K"]
    return {"bytes": n * (33 / 32 + (2 if case["type"] == "bf16" else 4)), "flops": 3 * n}


# ------------------------------------------------------------------------------- the definitions in 64 bits
def _exact_select(case, st):
    """Row by row orders from numpy's stable sorts, on the host."""
    l = st["logits"].cpu().numpy().astype(np.float64)
    T, E = l.shape
    G, M, k = case["groups"], case["kept"], case["k"]
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if case["scoring"] == "sigmoid":
            s = np.where(l >= 0, 1.0 / (1.0 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1.0 + np.exp(-np.abs(l))))
        else:
            top = l.max(1, keepdims=True)
            s = np.where(np.isfinite(l), np.exp(l - np.where(np.isfinite(top), top, 0.0)), 0.0)
            s /= np.where(s.sum(1, keepdims=True) > 0, s.sum(1, keepdims=True), 1.0)
    off = ~np.isfinite(l)
    c = s if st["b"] is None else s + st["b"].cpu().numpy().astype(np.float64)
    order = np.where(off, np.inf, -(l if st["b"] is None else c))
    dropped = np.zeros((T, G), dtype=bool)
    if G > 1:
        part = np.sort(np.where(off, -np.inf, c).reshape(T, G, E // G), axis=2)[:, :, ::-1]
        score = part[:, :, 0].copy()
        if case["by"] == "top2" and E // G > 1:
            score += np.where(np.isinf(part[:, :, 1]), 0.0, part[:, :, 1])
        np.put_along_axis(dropped, np.argsort(-score, axis=1, kind="stable")[:, M:], True, axis=1)
    dropped = np.repeat(dropped, E // G, axis=1)
    # three keys: groups that stay, experts that are not shut off, then the score; ties to the lower index
    first = np.argsort(order, axis=1, kind="stable")
    late = np.take_along_axis(dropped, first, 1) * 2 + np.take_along_axis(off, first, 1)
    idx = np.take_along_axis(first, np.argsort(late, axis=1, kind="stable"), 1)[:, :k]
    w = np.take_along_axis(s, idx, 1)
    if case["renorm"]:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return {"idx": torch.from_numpy(idx.astype(np.int32)), "w": torch.from_numpy(w * case["scale"])}


def _exact_codes(v):
    """Unrounded quotients in place of the codes; the scales are whole powers of two."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    s = torch.ceil(torch.log2(b.abs().amax(-1) / 448.0)).clamp(-127, 127)
    return (b * torch.exp2(-s).unsqueeze(-1)).reshape(v.shape)


def exact(case, seed):
    st = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "select":
        return _exact_select(case, st)
    if case["op"] == "select_grad":
        l, idx, dw = st["logits"].to(f8), st["idx"].long(), st["dw"].to(f8) * case["scale"]
        chosen = torch.zeros_like(l).scatter_(1, idx, 1.0)
        up = torch.zeros_like(l).scatter_(1, idx, dw)
        alive = l > -math.inf
        logp = torch.nn.functional.logsigmoid(l) if case["scoring"] == "sigmoid" else l
        if case["renorm"] or case["scoring"] == "softmax":
            over = (chosen > 0) & alive if case["renorm"] else alive
            z = torch.where(over, logp, -math.inf)
            z = z - torch.where(over.any(1, keepdim=True), z.amax(1, keepdim=True), 0.0)
            p = torch.where(over, torch.exp(z), 0.0)
            p = p / torch.where(over.any(1, keepdim=True), p.sum(1, keepdim=True), 1.0)
            dz = p * (up - torch.einsum("te,te->t", p, up).unsqueeze(1))
            dl = dz * torch.sigmoid(-l) if case["scoring"] == "sigmoid" else dz
        else:
            dl = up * torch.sigmoid(l) * torch.sigmoid(-l)
        dl = torch.where(alive, dl, 0.0)
        return dl if st["daux"] is None else dl + st["daux"].to(f8)
    if case["op"] in ("sandwich", "sandwich_grad"):
        d = case["d"]
        x = (_wide(tuple(_typed_pair(st["x"]))) if case.get("packed") else st["x"]).to(f8)
        W = st["post"].to(f8) * (1.0 if st["cg"] is None else st["cg"].to(f8))
        t = torch.ones(case["T"], dtype=f8, device="cuda") if st["tg"] is None else st["tg"].to(f8)
        rx = (torch.linalg.vector_norm(x, dim=1).square() / d + EPS) ** -0.5
        if case["op"] == "sandwich":
            h = torch.einsum("td,d,t->td", x, W, rx * t).add_(st["r"], alpha=RES_SCALE)
            out = {"residual": h}
            if case["next"]:
                rh = (torch.linalg.vector_norm(h, dim=1).square() / d + EPS) ** -0.5
                out["y"] = torch.einsum("td,d,t->td", h, st["w"].to(f8), rh)
                if case["mx"]:
                    out["codes"], out["scales"] = _exact_codes(out["y"]), None
            if case["save"]:
                out["x_codes"], out["x_scales"] = _exact_codes(x), None
                out["h_codes"], out["h_scales"] = _exact_codes(h), None
            return out
        out, ds = {}, torch.zeros_like(x) if st["dres"] is None else st["dres"].to(f8)
        if case["next"]:
            h = (_wide(tuple(_typed_pair(st["h"]))) if case["packed"] else st["h"]).to(f8)
            dy = st["dy"].to(f8)
            g = dy * st["w"].to(f8)
            rh = (torch.linalg.vector_norm(h, dim=1).square() / d + EPS) ** -0.5
            dot = torch.einsum("td,td->t", g, h) / d
            ds = ds + g * rh.unsqueeze(1) - h * (dot * rh ** 3).unsqueeze(1)
            out["dweight"] = torch.einsum("td,td,t->d", dy, h, rh)
            del h, dy, g
        q = torch.einsum("td,td,d,t->t", ds, x, W, rx)
        a = torch.einsum("td,td,t->d", ds, x, rx * t)
        out["dx"] = ds * W * (rx * t).unsqueeze(1) - x * (q * rx * rx * t / d).unsqueeze(1)
        out["dresidual"] = RES_SCALE * ds
        out["dpost_weight"] = a if st["cg"] is None else a * st["cg"].to(f8)
        if st["cg"] is not None:
            out["dgate"] = a * st["post"].to(f8)
        if st["tg"] is not None:
            out["dtoken_gate"] = q
        return out
    if case["op"] == "pack":
        return {"codes": _exact_codes(st["x"].to(f8)), "scales": None}
    codes, scales = _typed_pair((st["codes"], st["scales"]))
    return torch.ldexp(codes.to(f8).view(*scales.shape, 32), (scales.view(torch.uint8).int() - 127).unsqueeze(-1)).view(
        codes.shape)


def _typed_pair(packed):
    return packed[0].view(torch.float8_e4m3fn), packed[1].view(torch.float8_e8m0fnu)
