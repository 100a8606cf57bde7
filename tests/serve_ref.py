"""Plain 64-bit forms of the operators of a step over many requests, for the
tests: numpy, written from the definitions in include/mmvq_serve.h."""
from __future__ import annotations

import numpy as np

from quantized_decode_gemv_quantize_amd import binding as B

BLOCK = {B.Q4_0: (32, 18), B.Q4_1: (32, 20), B.Q5_0: (32, 22), B.Q5_1: (32, 24), B.Q8_0: (32, 34), B.Q4_K: (256, 144),
         B.Q5_K: (256, 176), B.Q6_K: (256, 210)}
FLOATS = {B.F32: 4, B.F16: 2, B.BF16: 2}
U = 2.0 ** -24                                  # a rounding to fp32


# --- tables ----------------------------------------------------------------------

def _block(b, kind):
    """Values of one block of bytes."""
    half = lambda at: float(np.frombuffer(b[at:at + 2].tobytes(), np.float16)[0])
    v, i8 = np.zeros(BLOCK[kind][0]), b.view(np.int8)
    if kind == B.Q8_0:
        return half(0) * i8[2:].astype(np.float64)
    if kind == B.Q6_K:
        for h in range(2):
            for l in range(32):
                ql, qk, qh = int(b[64 * h + l]), int(b[64 * h + 32 + l]), int(b[128 + 32 * h + l])
                for g, low in enumerate((ql & 15, qk & 15, ql >> 4, qk >> 4)):
                    q = low + 16 * (qh >> (2 * g) & 3) - 32
                    v[128 * h + 32 * g + l] = half(208) * int(i8[192 + 8 * h + 2 * g + l // 16]) * q
        return v
    if kind in (B.Q4_K, B.Q5_K):
        s = [int(x) for x in b[4:16]]
        for t in range(8):
            sc, m = (s[t] & 63, s[t + 4] & 63) if t < 4 else ((s[t + 4] & 15) | s[t - 4] >> 6 << 4, s[t + 4] >> 4 | s[t] >> 6 << 4)
            for l in range(32):
                q = int(b[(16 if kind == B.Q4_K else 48) + 32 * (t // 2) + l]) >> (4 * (t % 2)) & 15
                if kind == B.Q5_K:
                    q += 16 * (int(b[16 + l]) >> t & 1)
                v[32 * t + l] = half(0) * sc * q - half(2) * m
        return v
    codes = BLOCK[kind][1] - 16
    fifth = int.from_bytes(b[codes - 4:codes].tobytes(), "little") if kind in (B.Q5_0, B.Q5_1) else 0
    for j in range(32):
        q = (int(b[codes + j % 16]) >> (4 * (j // 16)) & 15) + 16 * (fifth >> j & 1)
        v[j] = half(0) * q + half(2) if kind in (B.Q4_1, B.Q5_1) else half(0) * (q - (16 if kind == B.Q5_0 else 8))
    return v


def table_row(row, kind):
    """Values of a table's row of bytes."""
    if kind == B.F32:
        return row.view(np.float32).astype(np.float64)
    if kind == B.F16:
        return row.view(np.float16).astype(np.float64)
    if kind == B.BF16:
        return (row.view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return np.concatenate([_block(b, kind) for b in row.reshape(-1, BLOCK[kind][1])])


def row_bytes(kind, K):
    return K * FLOATS[kind] if kind in FLOATS else K // BLOCK[kind][0] * BLOCK[kind][1]


# --- pages -----------------------------------------------------------------------

class Pool:
    """A pool's state on the host; release() and plan() are the definitions."""

    def __init__(self, n_seqs, pages_per_seq, n_pages, page, n_free, rng, held=None):
        self.page, self.n_pages, self.wide = page, n_pages, pages_per_seq
        order = rng.permutation(n_pages).astype(np.int32)
        self.free, self.n_free = np.full(n_pages, -7, dtype=np.int32), n_free
        self.free[:n_free] = order[:n_free]
        self.table = np.full((n_seqs, pages_per_seq), -1, dtype=np.int32)
        self.held = np.zeros(n_seqs, dtype=np.int32) if held is None else np.asarray(held, dtype=np.int32)
        at = n_free
        for s in range(n_seqs):
            self.table[s, :self.held[s]] = order[at:at + self.held[s]]
            at += self.held[s]
        assert at <= n_pages

    def release(self, keep, shared=None):
        for s in range(len(self.held)):
            held = min(max(int(self.held[s]), 0), self.wide)
            if not 0 <= keep[s] < held:
                continue
            for p in range(keep[s], held):
                page = self.table[s, p]
                if 0 <= page < self.n_pages and (shared is None or p >= shared[s]) and self.n_free < self.n_pages:
                    self.free[self.n_free] = page
                    self.n_free += 1
                self.table[s, p] = -1
            self.held[s] = keep[s]

    def plan(self, cached, new, n_rows):
        n, page = len(self.held), self.page
        start, length, wanted = [0], [], []
        for s in range(n):
            c, k = min(max(int(cached[s]), 0), 1 << 30), min(max(int(new[s]), 0), n_rows - start[-1])
            start.append(start[-1] + k)
            length.append(c + k)
            if k > 0:
                wanted += [(s, p) for p in range(self.held[s], min(-(-(c + k) // page), self.wide))]
        g = min(len(wanted), self.n_free)
        for i, (s, p) in enumerate(wanted):
            self.table[s, p] = self.free[self.n_free - g + i] if i < g else -1
            self.held[s] += i < g
        self.n_free -= g
        seq, pos, slot = np.full(n_rows, -1, np.int32), np.full(n_rows, -1, np.int32), np.full(n_rows, -1, np.int64)
        for s in range(n):
            for r in range(start[s], start[s + 1]):
                seq[r], pos[r] = s, length[s] - (start[s + 1] - r)
                p = pos[r] // page
                if p < self.wide and 0 <= self.table[s, p] < self.n_pages:
                    slot[r] = int(self.table[s, p]) * page + pos[r] % page
        return np.array(start, np.int32), np.array(length, np.int32), seq, pos, slot, len(wanted) - g


# --- adapters --------------------------------------------------------------------

def lora(A, Bw, ranks, scales, x, base, ids, parts):
    """Values in 64 bits, and how far fp32 sums may be off. A product of 32
    values a matrix instruction: its own sum is off by 32 U of its terms'
    magnitudes, what it is added to by a rounding of the sum so far; an
    instruction a part (3, 6 or 8) and step of 32, the longest chain one wave's
    quarter of a range or all ranks, then 4 waves and 16 ranges; three roundings
    at the end. Products of parts are exact to 2^-28."""
    out, tol = base.astype(np.float64), 3 * U * np.abs(base).astype(np.float64)
    instr = {1: 3, 2: 6, 3: 8}[parts]
    for t, a in enumerate(ids):
        if a < 0:
            tol[t] = 0.0
            continue
        r = min(max(int(ranks[a]), 0), A.shape[1])
        a64, b64, x64 = A[a, :r].astype(np.float64), Bw[a][:, :r].astype(np.float64), x[t].astype(np.float64)
        v, mag = a64 @ x64, np.abs(a64) @ np.abs(x64)
        steps = -(-A.shape[2] // 32)
        dv = U * (32 + instr * (-(-steps // 4)) + 20 + 1) * mag
        y, most = b64 @ v, np.abs(b64) @ np.abs(v)
        dy = np.abs(b64) @ dv + U * (32 + instr * (-(-r // 32)) + 1) * most
        out[t] += float(scales[a]) * y
        tol[t] += abs(float(scales[a])) * (dy + 3 * U * most)
    return out, tol


# --- sampling --------------------------------------------------------------------

def distribution(z, T=1.0, k=0, p=1.0, m=0.0):
    """Kept weights of a row of logits, in 64 bits."""
    z = np.where(np.isnan(z), -np.inf, z.astype(np.float64))
    top, V = z.max(), len(z)
    if top == -np.inf:
        return np.zeros(V)
    if not T > 0:
        return (np.arange(V) == z.argmax()).astype(np.float64)
    if top == np.inf:
        w = (z == np.inf).astype(np.float64)
    else:
        with np.errstate(invalid="ignore"):
            w = np.where(z == -np.inf, 0.0, np.exp(np.where(z == -np.inf, 0.0, z - top) / float(np.float32(T))))
    order = np.lexsort((np.arange(V), -z))
    order = order[z[order] > -np.inf]
    if 0 < k < V:
        order = order[:k]
    if p < 1:
        before = np.concatenate([[0.0], np.cumsum(w[order])[:-1]])
        n = int((before < float(np.float32(p)) * w[order].sum()).sum())
        order = order[:max(n, 1)]
    if m > 0:
        order = order[w[order] >= min(float(np.float32(m)), 1.0)]
    kept = np.zeros(V)
    kept[order] = w[order]
    return kept


def drawn(w, u):
    if not w.sum() > 0:
        return -1
    up = np.cumsum(w)
    hit = np.flatnonzero(up > float(u) * up[-1])
    return int(hit[0]) if len(hit) else int(np.flatnonzero(w > 0)[-1])
