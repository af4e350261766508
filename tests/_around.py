"""Plain 64-bit forms of the operators around the layer (numpy), for the tests.  They share no
code with the library."""

import numpy as np


def rms_norm(x, w, eps, r=None):
    h = x if r is None else x + r
    return h * (1.0 / np.sqrt((h * h).mean(1, keepdims=True) + eps)) * w, h


def rms_norm_grad(dy, s, w, eps, dres=None):
    rho = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    xhat, g = s * rho, dy * w
    ds = rho * (g - xhat * (g * xhat).mean(1, keepdims=True))
    return (ds if dres is None else ds + dres), (dy * xhat).sum(0)


def mx_exponents(v):
    """Smallest s with amax <= 448 * 2^s for each block of 32 along the last axis (-127 for 0)."""
    amax = np.abs(v.reshape(*v.shape[:-1], -1, 32)).max(-1)
    with np.errstate(divide="ignore"):
        s = np.ceil(np.log2(amax / 448.0))
    return np.where(amax > 0, np.clip(s, -127, 127), -127), amax


def e4m3(codes):
    """Values of E4M3 code bytes."""
    c = np.asarray(codes, dtype=np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m * 2.0 ** -9)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def sequences(T, offsets, mask):
    """Sequence of every token, -1 for those left out."""
    seq = np.zeros(T, dtype=np.int64) if offsets is None else np.full(T, -1)
    if offsets is not None:
        for s, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])):
            seq[a:b] = s
    if mask is not None:
        seq[~mask] = -1
    return seq


def balance(logits, idx, S, seq, alpha, z_coef):
    """loss [2], counts [S,E], dlogits; tokens with seq < 0 do not exist."""
    T, E = logits.shape
    k = idx.shape[1]
    ok = seq >= 0
    n = max(1, int(ok.sum()))
    counts = np.zeros((S, E), dtype=np.int64)
    for t in np.nonzero(ok)[0]:
        for e in idx[t]:
            if 0 <= e < E:
                counts[seq[t], e] += 1
    n_seq = np.bincount(seq[ok], minlength=S)
    dl, loss = np.zeros((T, E)), [0.0, 0.0]
    for t in np.nonzero(ok)[0]:
        l = logits[t]
        top = l.max()
        if top == -np.inf:
            continue
        e = np.exp(l - top)
        p, lse = e / e.sum(), top + np.log(e.sum())
        c = counts[seq[t]]
        a = alpha * E / (k * n * n_seq[seq[t]])
        inner = (c * p).sum()
        loss[0] += a * inner
        loss[1] += z_coef / n * lse * lse
        dl[t] = p * (a * (c - inner) + 2 * z_coef / n * lse)
    return np.array(loss), counts, dl


def adamw(w, g, m, v, lr, b1, b2, eps, decay, step):
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    upd = (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps) + decay * w
    return w - lr * upd, m, v
