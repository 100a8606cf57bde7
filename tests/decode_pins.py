"""Inputs at which the precision of the attention operator's two-part products
shows, and bounds that a form with fewer bits does not keep.

Keys have one value each, so that a score is one product whatever the head's
size, and a row sees three of them: nothing averages errors out."""
import numpy as np

import decode_ref as R

WINDOW, BASE = 3, 20


def inputs(kind, D, part, new, H=2, G=4):
    """k, v [tokens, H, D] and q [new, H G, D], fp32. part "q": scores of 23 to
    29 that differ by the query's own bits; "weights": scores within 1 of each
    other, and values so small that no exponent joins the scores."""
    rng = np.random.default_rng(D * 10 + new)
    n = new + BASE
    k = np.zeros((n, H, D), np.float32)
    k[np.arange(n)[:, None], np.arange(H), rng.integers(0, D, (n, H))] = 1.0
    v = rng.standard_normal((n, H, D))
    if part == "q":
        q = 26.0 * (1 + 0.04 * np.clip(rng.standard_normal((new, H * G, D)), -3, 3))
    else:
        q = rng.uniform(-0.5, 0.5, (new, H * G, D))
        v *= 2.0 ** -13
    return k, v.astype(np.float32), (q * D ** 0.5).astype(np.float32)


def tolerance(mag, part, v):
    """Score: the query in two parts (2^-21 of the row's largest value, which
    is at most 1.28 times any), three roundings of it (its scaling, the sum of
    the parts' products, the block's scale) and two of its sum with the
    exponent of a value's scale (below 22.2 = 32 ln 2 where values are
    ordinary, ln 2 where they are small). Probability: twice that, exp2 2^-22,
    its parts 2^-20, eight roundings of sums, join and quotient; 1.5 2^-33 of
    the largest value a key (decode_ref)."""
    size, exponent = (29.2, 22.2) if part == "q" else (0.51, 0.7)
    ds = size * (1.28 * 2.0 ** -21 + 3 * 2.0 ** -24) + 2 * (size + exponent) * 2.0 ** -24
    rel = 2 * np.expm1(ds) + 2.0 ** -22 + 2.0 ** -20 + 8 * 2.0 ** -24
    return rel * mag + WINDOW * 1.5 * 2.0 ** -33 * np.abs(v).max()


def _bits(x, top, bits):
    """x to `bits` bits of `top` (of its own size where top is None)."""
    size = np.abs(x) if top is None else top
    unit = 2.0 ** (np.floor(np.log2(np.where(size == 0, 1.0, size))) + 1 - bits)
    return np.round(x / unit) * unit


def model(q, k, v, scale, q_bits, w_bits):
    """The operator in 64 bits but for a query of q_bits of its row's largest
    value and weights of w_bits where they meet the values."""
    n, heads, D = q.shape
    G = heads // k.shape[1]
    q = _bits(q.astype(np.float64), np.abs(q).max(-1, keepdims=True).astype(np.float64), q_bits)
    out = np.zeros(q.shape)
    key, pos = np.arange(len(k))[None], BASE + np.arange(n)[:, None]
    see = (key <= pos) & (key > pos - WINDOW)
    for h in range(heads):
        z = np.where(see, scale * (q[:, h] @ k[:, h // G].T), -np.inf)
        w = np.exp(z - z.max(-1, keepdims=True))
        out[:, h] = _bits(w, None, w_bits) @ v[:, h // G] / w.sum(-1, keepdims=True)
    return out


def reference(q, k, v, scale):
    ref, mag, _ = R.attention(q, k, v, scale, BASE, WINDOW)
    return ref, mag
