"""Plain 64-bit forms of the operators of a block (numpy), for the tests.  They share no code with
the library."""

import numpy as np

SHUT = -1e30


def scores(l, scoring):
    """softmax or sigmoid along the last axis; logits at or below -1e30 and NaN have none."""
    l = np.asarray(l, dtype=np.float64)
    on = l > SHUT
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            return np.where(on, 1.0 / (1.0 + np.exp(-np.where(on, l, 0.0))), 0.0)
        top = np.max(np.where(on, l, -np.inf), axis=-1, keepdims=True)
        e = np.where(on, np.exp(np.where(l == top, 0.0, np.where(on, l, 0.0) - np.where(np.isfinite(top), top, 0.0))), 0.0)
        e = np.where(on & np.isposinf(top) & (l != top), 0.0, e)
    total = e.sum(-1, keepdims=True)
    return e / np.where(total > 0, total, 1.0)


def select(logits, k, scoring, bias=None, groups=1, kept=1, by="max", renorm=True, scale=1.0):
    """(idx, w): token by token, by sorting tuples."""
    T, E = logits.shape
    s = scores(logits, scoring)
    idx, w = np.zeros((T, k), dtype=np.int64), np.zeros((T, k))
    n = E // groups
    for t in range(T):
        shut = ~(logits[t].astype(np.float64) > SHUT)
        c = s[t].copy()
        if bias is not None:
            b = bias.astype(np.float64)
            shut = shut | ~(np.abs(b) < 1e30)
            c = c + np.where(shut, 0.0, b)
        order = c if bias is not None else logits[t].astype(np.float64)
        open_ = [[c[e] for e in range(g * n, g * n + n) if not shut[e]] for g in range(groups)]
        score = [sum(sorted(v)[-2:]) if by == "top2" and v else max(v, default=-np.inf) for v in open_]
        stay = sorted(range(groups), key=lambda g: (-score[g], g))[:kept]
        pool = [e for g in stay for e in range(g * n, g * n + n)]
        pool.sort(key=lambda e: (shut[e], 0.0 if shut[e] else -order[e], e))
        idx[t] = pool[:k]
        w[t] = s[t, idx[t]]
        if renorm:
            w[t] = w[t] / w[t].sum() if w[t].sum() > 0 else 0.0
    return idx, w * scale


def select_grad(logits, idx, dw, scoring, renorm=True, scale=1.0):
    T, E = logits.shape
    s = scores(logits, scoring)
    out = np.zeros((T, E))
    for t in range(T):
        ok = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
        sj = np.array([s[t, idx[t, j]] for j in ok])
        d = dw[t, ok] * scale
        if renorm:
            p = sj / sj.sum() if sj.sum() > 0 else 0.0 * sj
            g = p * (d - (p * d).sum()) * (1.0 - sj if scoring == "sigmoid" else 1.0)
        elif scoring == "sigmoid":
            g = sj * (1.0 - sj) * d
        else:
            out[t] -= s[t] * (sj * d).sum()
            g = sj * d
        for j, v in zip(ok, g):
            out[t, idx[t, j]] += v
    return out


def sandwich(x, r, post, weight=None, gate=None, token_gate=None, a=1.0, eps=1e-6):
    """(h, v)."""
    n = x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * post
    n = n * (1.0 if gate is None else gate) * (1.0 if token_gate is None else token_gate[:, None])
    h = a * r + n
    return h, None if weight is None else h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight


def sandwich_grad(x, h, post, dy=None, dres=None, weight=None, gate=None, token_gate=None, a=1.0, eps=1e-6):
    out, ds = {}, np.zeros_like(x) if dres is None else dres
    if dy is not None:
        rho = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
        hhat, g = h * rho, dy * weight
        ds = ds + rho * (g - hhat * (g * hhat).mean(1, keepdims=True))
        out["dweight"] = (dy * hhat).sum(0)
    W = post if gate is None else post * gate
    t = np.ones((len(x), 1)) if token_gate is None else token_gate[:, None]
    rho = 1.0 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    xhat, gw = x * rho, ds * W
    A = (t * ds * xhat).sum(0)
    out.update(dx=rho * t * (gw - xhat * (gw * xhat).mean(1, keepdims=True)), dresidual=a * ds,
               dpost_weight=A * (1.0 if gate is None else gate))
    if gate is not None:
        out["dgate"] = A * post
    if token_gate is not None:
        out["dtoken_gate"] = (gw * xhat).sum(1)
    return out
