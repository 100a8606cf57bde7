"""Plain 64-bit forms of the operators between the mat-vecs, for the tests:
numpy, written from the definitions in include/mmvq_decode.h, and builders
of ragged paged batches."""
from __future__ import annotations

import numpy as np

from quantized_decode_gemv_quantize_amd import binding as B

KINDS = {"f16": B.F16, "q8_0": B.Q8_0, "q4_0": B.Q4_0}


def f32(x):
    return np.asarray(x).astype(np.float32).astype(np.float64)


# --- stored values -----------------------------------------------------------

def q8_codes(x):
    """Codes and fp16 scales of [..., 32] values by the q8 rule: scale and
    quotient are fp32 (the 64-bit product and quotient of fp32 values rounded
    to fp32 are the fp32 ones), roundf goes away from zero."""
    x = np.asarray(x, dtype=np.float64)
    d = f32(np.abs(x).max(-1, keepdims=True) * float(np.float32(1.0) / np.float32(127.0)))
    safe = np.where(d == 0, 1.0, d)
    t = f32(x / safe)
    q = np.where(d == 0, 0.0, np.copysign(np.floor(np.abs(t) + 0.5), t))
    return q, d.astype(np.float16)


def q4_codes(x):
    """Codes (less 8) and fp16 scales of [..., 32] values by the q4 rule."""
    x = np.asarray(x, dtype=np.float64)
    most = np.take_along_axis(x, np.abs(x).argmax(-1)[..., None], -1)
    d = most / -8.0
    safe = np.where(d == 0, 1.0, d)
    q = np.clip(np.floor(f32(f32(x / safe) + 8.5)), 0, 15)
    return np.where(d == 0, 8.0, q) - 8.0, d.astype(np.float16)


def stored(x, kind):
    """What a cache of this type holds of fp32 values [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    if kind == "f16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(np.float64)
    blk = x.reshape(*x.shape[:-1], -1, 32)
    q, d = q8_codes(blk) if kind == "q8_0" else q4_codes(blk)
    return (q * d.astype(np.float64)).reshape(x.shape)


# --- norm ----------------------------------------------------------------------

def rms_norm(x, res, w, eps):
    h = x.astype(np.float64) if res is None else f32(x.astype(np.float64) + res)
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + float(np.float32(eps)))
    return h, y if w is None else y * w.astype(np.float64)


# --- paged batches ---------------------------------------------------------------

class Paged:
    """A ragged batch over a cache: news[s] new tokens of lens[s] in all."""

    def __init__(self, kind, D, H, page, news, lens, seed=0, extra_rows=(0, 0), spare=2, fill=0xA5):
        import torch
        rng = np.random.default_rng(seed)
        self.kind, self.D, self.H, self.page, self.news, self.lens = kind, D, H, page, list(news), list(lens)
        need = [max(1, -(-l // page)) for l in lens]
        self.n_pages, self.wide = sum(need) + spare, max(need)
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), self.wide), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.start = (np.concatenate([[0], np.cumsum(news)]) + extra_rows[0]).astype(np.int32)
        self.n_tokens = int(self.start[-1]) + extra_rows[1]
        self.page_bytes = B.mmvq_kv_page_bytes(KINDS[kind], page, H, D)
        self.k = torch.full((self.n_pages, self.page_bytes), fill, dtype=torch.uint8, device="cuda:0")
        self.v = self.k.clone()
        self.upload()

    def upload(self):
        import torch
        self.d = [torch.from_numpy(a).to("cuda:0") for a in
                  (self.start, np.asarray(self.lens, dtype=np.int32), np.ascontiguousarray(self.table))]

    @property
    def cache(self):
        return B.kv_cache(self.k, self.v, KINDS[self.kind], self.n_pages, self.page, self.H, self.D)

    def batch(self, whole=False, max_new=None, max_len=None):
        """The new tokens, or every token of every sequence (rows of `whole` buffers)."""
        import torch
        if whole:
            start = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32)
            self.whole_start = torch.from_numpy(start).to("cuda:0")
            return B.kv_batch(self.whole_start, self.d[1], self.d[2], len(self.lens), int(start[-1]),
                              max(1, max(self.lens)), max(1, max(self.lens)), self.wide)
        return B.kv_batch(self.d[0], self.d[1], self.d[2], len(self.lens), self.n_tokens,
                          max_new or max(1, max(self.news)), max_len or max(1, max(self.lens)), self.wide)

    def fill(self, rng, scale=1.0):
        """Random keys and values for all tokens, written through the library; returns what is stored."""
        import torch
        total = sum(self.lens)
        raw = [(rng.standard_normal((total, self.H * self.D)) * scale).astype(np.float32) for _ in "kv"]
        dk, dv = (torch.from_numpy(r).to("cuda:0") for r in raw)
        if total:
            B.mmvq_kv_write(self.cache, self.batch(whole=True), dk, self.H * self.D, dv, self.H * self.D)
        at = np.concatenate([[0], np.cumsum(self.lens)])
        got = [stored(r.reshape(total, self.H, self.D), self.kind) for r in raw]
        return [[g[at[s]:at[s + 1]] for s in range(len(self.lens))] for g in got]


def attention(q, k, v, scale, base, window=0, sinks=None, hidden=()):
    """q [n, heads, D] at positions base.., k, v [keys, H, D] -> out, and the
    sums of |p v| and of |p v| weighted by |score error bounds| that tolerances use."""
    n, heads, D = q.shape
    keys, H, _ = k.shape
    G = heads // H
    out, mag, smax = np.zeros((n, heads, D)), np.zeros((n, heads, D)), np.zeros((n, heads))
    pos = base + np.arange(n)[:, None]
    key = np.arange(keys)[None]
    see = (key <= pos) & (key > pos - window if window else key >= 0)
    for t in hidden:
        see[:, t] = False
    for h in range(heads):
        kk, vv = k[:, h // G], v[:, h // G]
        z = np.where(see, 0.0, -np.inf)
        with np.errstate(invalid="ignore"):
            z = np.where(see, scale * (q[:, h].astype(np.float64) @ kk.T), -np.inf)
        # largest sum of |q k| a row meets: what the rounding of its scores goes by
        smax[:, h] = (np.where(see, abs(scale) * (np.abs(q[:, h]).astype(np.float64).max(-1, keepdims=True)
                                                  * np.abs(kk).sum(-1)[None]), 0.0)).max(-1, initial=0.0)
        top = z.max(-1, initial=-np.inf)
        if sinks is not None:
            top = np.where(np.isfinite(top), np.maximum(top, sinks[h]), top)
        live = np.isfinite(top)
        e = np.where(see, np.exp(np.where(see, z, 0.0) - np.where(live, top, 0.0)[:, None]), 0.0)
        total = e.sum(-1)
        if sinks is not None:
            total = total + np.where(live, np.exp(sinks[h] - np.where(live, top, 0.0)), 0.0)
        p = e / np.where(total > 0, total, 1.0)[:, None]
        out[:, h] = p @ np.where(see.any(0)[:, None], vv, 0.0)
        mag[:, h] = p @ np.where(see.any(0)[:, None], np.abs(vv), 0.0)
    return out, mag, smax


def attention_tolerance(out, mag, smax, v, D):
    """|gpu - ref| for fp32 results; v: the stored values [keys, H, D].
    Per score: q in two fp16 parts is off by 2^-21 of the row's largest |q|
    (smax has max|q| sum|k|), scaling it rounds once (2^-24), the products sum
    D terms in fp32 (D 2^-24 of sum|q k| <= smax), three more roundings of the
    score: ds <= smax (2^-21 + (D + 4) 2^-24). A probability moves by 2 ds
    (its own and the sum's) + 2^-22 (exp2), its two parts are off by 2^-20 at
    most, and the sums over the keys, 32 a step, round (keys/32 + 4 + 9)
    times: matrix products add 8 terms a lane group, 4 groups, 2 parts, then
    the joins.
    The two parts of p = 2^e m: the first, cut toward zero, leaves less than
    2^(e-10), which the second rounds by 2^(e-22). Of p d = 2^E M, where a
    scale joins, the first is off by 2^(E-11), the second holds that and less
    than p d 2^-10 / m of the rest: below 2^(E-9) its rounding is 2^(E-21);
    from there on, M >= 1.5 and it is 2^(E-20): 2^-20 / 1.5 of p d at most,
    together 0.92 2^-20.
    Below 2^-14 fp16 has steps of 2^-24. F16: a weight is off by 2^-25 where
    the largest is 2^10 at least. Quantized: by 2^-25 times a normalised scale
    below 4, and its product by 2^-25 twice more, 1.5 2^-23 together, where
    the largest weight is at least 2^9 and its scale 2: 1.5 2^-33 of the
    largest value a key, the code with the largest magnitude being in every
    block."""
    keys = max(1, len(v))
    ds = smax * (2.0 ** -21 + (D + 4) * 2.0 ** -24)
    with np.errstate(over="ignore"):
        rel = 2 * np.expm1(ds) + 2.0 ** -22 + 2.0 ** -20 + (keys / 32 * 2 + 48) * 2.0 ** -24
    low = 1.5 * 2.0 ** -33 * keys * np.abs(v).max(initial=0.0)
    return mag * rel[..., None] + np.abs(out) * 2.0 ** -23 + low + 1e-30


# --- verification ------------------------------------------------------------------

def verify(target, kind, temp, tok, dp, start, ua, us, wide):
    count = np.zeros(len(start) - 1, dtype=np.int32)
    out = np.full((len(start) - 1, wide), -1, dtype=np.int32)

    def put(s, i, t):
        if i < wide:
            out[s, i] = t

    for s in range(len(start) - 1):
        for r in range(start[s], start[s + 1]):
            row = target[r].astype(np.float64)
            if kind == B.TARGET_LOGITS:
                row = np.where(np.isnan(row), -np.inf, row)
                top = row.max()
                T = 1.0 if temp is None else float(temp[s])
                if top == -np.inf:
                    p = np.zeros(len(row))
                elif not T > 0:
                    p = (np.arange(len(row)) == row.argmax()).astype(np.float64)
                elif top == np.inf:
                    p = (row == np.inf).astype(np.float64)
                else:
                    with np.errstate(invalid="ignore"):
                        p = np.where(row == -np.inf, 0.0, np.exp((row - top) * (1.0 / T)))
            else:
                p = np.where((row > 0) & (row < np.inf), row, 0.0)
            z = p.sum()
            if not z > 0:
                break
            p = p / z
            if r + 1 < start[s + 1]:
                x = int(tok[r])
                if dp is not None:
                    q = np.where(dp[r] > 0, dp[r].astype(np.float64), 0.0)
                else:
                    q = (np.arange(len(p)) == x).astype(np.float64)
                if 0 <= x < len(p) and float(ua[r]) * q[x] < p[x]:
                    put(s, count[s], x)
                    count[s] += 1
                    continue
                left = np.maximum(p - q, 0.0)
                p = left if left.sum() > 0 else p
            up = np.cumsum(p)
            hit = np.nonzero(up > float(us[s]) * up[-1])[0]
            put(s, count[s], hit[0] if len(hit) else np.nonzero(p)[0][-1])
            break
    return count, out
