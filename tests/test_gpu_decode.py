"""Operators between the mat-vecs on the GPU, against plain 64-bit forms:
the residual RMS norm with q8_1 output, the paged cache's writer and reader,
attention over the cache, and the verification of drafted tokens."""
import numpy as np
import pytest

import decode_ref as R
from gpu_helpers import announce, dev, host
from quantized_decode_gemv_quantize_amd import binding as B

pytestmark = pytest.mark.gpu

EPS = 1e-5
HALF32 = 2.0 ** -24


def nan(*shape):
    import torch
    return torch.full(shape, float("nan"), device="cuda:0")


def d32(blk):
    """fp32 scales of [..., 32] values, before they are stored as fp16."""
    return R.f32(np.abs(blk.astype(np.float64)).max(-1, keepdims=True) * float(np.float32(1.0) / np.float32(127.0)))


# --- norm -------------------------------------------------------------------------

@pytest.mark.parametrize("n,K,ldx,off", [
    (1, 32, 32, 0), (3, 96, 100, 1), (1, 4096, 4096, 0), (5, 4128, 4131, 1), (2, 1024, 1024, 0), (7, 2048, 2052, 3),
    (2, 8192, 8192, 0), (3, 14336, 14336, 0), (2, 16384, 16384, 0), (2, 16416, 16417, 1), (1, 40000, 40000, 0), (300, 64, 64, 0)])
def test_norm_q8_1(n, K, ldx, off):
    import torch
    announce(f"norm n={n} K={K} ldx={ldx} off={off}")
    rng = np.random.default_rng(n * 1000 + K)
    x, r = (rng.standard_normal((n, ldx)).astype(np.float32) * s for s in (1.0, 3.0))
    w = (1 + 0.3 * rng.standard_normal(K)).astype(np.float32)
    flat = [dev(np.concatenate([np.zeros(off, np.float32), a.reshape(-1)])) for a in (x, r)]
    xd, rd = flat[0][off:], flat[1][off:]
    h, y = nan(n, ldx), nan(n, ldx)
    yq = torch.full((n, K // 32 * 36), 0xA5, dtype=torch.uint8, device="cuda:0")
    B.mmvq_add_rms_norm(xd, K, n, ldx, rd, ldx, dev(w), EPS, h, ldx, y, ldx, yq)
    eh, ey = R.rms_norm(x[:, :K], r[:, :K], w, EPS)
    gh, gy = host(h), host(y)
    assert np.array_equal(gh[:, :K].astype(np.float64), eh)
    # one rounding to fp32 of a value that is off by some 2^-50
    assert (np.abs(gy[:, :K] - ey) <= np.abs(ey) * HALF32 * (1 + 1e-6)).all()
    assert np.isnan(gh[:, K:]).all() and np.isnan(gy[:, K:]).all()
    q, d = R.q8_codes(gy[:, :K].astype(np.float64).reshape(n, -1, 32))
    with np.errstate(over="ignore"):
        s = R.f32(d32(gy[:, :K].reshape(n, -1, 32)) * q.sum(-1, keepdims=True)).astype(np.float16)
    want = np.concatenate([d.view(np.uint8), s.view(np.uint8), q.astype(np.int8).view(np.uint8)], -1).reshape(n, -1)
    assert np.array_equal(host(yq), want)
    alone = torch.zeros_like(yq)                     # q8_1 only, no sum stored
    B.mmvq_add_rms_norm(xd, K, n, ldx, rd, ldx, dev(w), EPS, None, 0, None, 0, alone)
    assert torch.equal(alone, yq)
    back = nan(n, K + 3)
    B.mmvq_dequantize_q8_1(yq, K, n, back, K + 3)
    assert np.array_equal(host(back)[:, :K], (q * d.astype(np.float64)).reshape(n, K).astype(np.float32))
    assert np.isnan(host(back)[:, K:]).all()


@pytest.mark.parametrize("n,K", [(1, 1), (4, 3), (2, 1999), (3, 4097), (2, 16385), (1, 33331)])
def test_norm_plain_lengths(n, K):
    rng = np.random.default_rng(K)
    x = rng.standard_normal((n, K)).astype(np.float32)
    y = nan(n, K + 2)
    B.mmvq_add_rms_norm(dev(x), K, n, K, None, 0, None, EPS, None, 0, y, K + 2, None)
    _, e = R.rms_norm(x, None, None, EPS)
    assert (np.abs(host(y)[:, :K] - e) <= np.abs(e) * HALF32 * (1 + 1e-6)).all() and np.isnan(host(y)[:, K:]).all()


@pytest.mark.parametrize("K", [4096, 20000])
@pytest.mark.parametrize("alias", ["x", "residual", "y"])
def test_norm_in_place(K, alias):
    rng = np.random.default_rng(K)
    x, r = (rng.standard_normal((3, K)).astype(np.float32) for _ in "ab")
    xd, rd, y = dev(x), dev(r), nan(3, K)
    s = {"x": xd, "residual": rd, "y": None}[alias]
    if alias == "y":
        y = xd
    B.mmvq_add_rms_norm(xd, K, 3, K, rd, K, None, EPS, s, K, y, K, None)
    eh, e = R.rms_norm(x, r, None, EPS)
    if s is not None:
        assert np.array_equal(host(s).astype(np.float64), eh)
    assert (np.abs(host(y) - e) <= np.abs(e) * HALF32 * (1 + 1e-6)).all()


def test_norm_extreme_values():
    """Zero columns give zeros, columns whose squares pass fp32 stay finite,
    and a NaN stays in its own column."""
    x = np.zeros((4, 256), np.float32)
    x[1] = 3e30
    x[2] = 1e-30
    x[3, 7] = np.nan
    y = nan(4, 256)
    B.mmvq_add_rms_norm(dev(x), 256, 4, 256, None, 0, None, EPS, None, 0, y, 256, None)
    g = host(y)
    _, e = R.rms_norm(x[:3], None, None, EPS)
    assert (g[0] == 0).all() and np.isnan(g[3]).all()
    assert (np.abs(g[:3] - e) <= np.abs(e) * HALF32 * (1 + 1e-6)).all()


# --- cache -------------------------------------------------------------------------

def unit_bytes(kind, D, keys, tt, d):
    """Bytes of a unit that hold dim d of token tt, and which part of them."""
    NB, b, c = D // 32, d // 32, d % 32
    run = {"f16": 16, "q8_0": 8, "q4_0": 4}[kind]
    if keys:
        g, off = (c % 16 // 4, b * run + c % 4) if kind == "q4_0" else (c // 8, b * run + c % 8 * (2 if kind == "f16" else 1))
        ps = next(p for p in (16, 8, 4) if run * NB % p == 0)
        return (((tt // 4 % 2 * (run * NB // ps) + off // ps) * 4 + g) * 8 + tt // 8 * 4 + tt % 4) * ps + off % ps
    if kind == "f16":
        return ((((b * 2 + c // 16) * 2 + tt // 8) * 16 + c % 16) * 8 + tt % 8) * 2
    if kind == "q8_0":
        return (((b * 2 + tt // 8) * 16 + c % 16) * 2 + c // 16) * 8 + tt % 8
    return ((b * 2 + tt // 8) * 16 + c % 16) * 8 + tt % 8


@pytest.mark.parametrize("kind", list(R.KINDS))
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_cache_round_trip(kind, D, page):
    """Ragged new tokens that start and end inside units and pages: stored
    values, the bytes of every other slot untouched, rows outside untouched."""
    announce(f"cache {kind} D={D} page={page}")
    H, news, lens = 3, [1, 0, 37, 16, 5, 50], [1, 9, 40, 32, 77, 65]
    p = R.Paged(kind, D, H, page, news, lens, seed=D + page, extra_rows=(2, 3))
    rng = np.random.default_rng(D)
    ld = 3 * H * D + 1
    act = rng.standard_normal((p.n_tokens, ld)).astype(np.float32) * np.exp(rng.standard_normal((p.n_tokens, 1))).astype(np.float32)
    act[3, :32] = 0                                     # a block of zeros
    act[4, 32:64] = 2.5                                 # equal magnitudes: the first decides
    act[4, 40] = -2.5
    ad = dev(act)
    B.mmvq_kv_write(p.cache, p.batch(), ad[:, H * D:], ld, ad[:, 2 * H * D:], ld)
    ko, vo = nan(p.n_tokens, H * D), nan(p.n_tokens, H * D + 5)
    B.mmvq_kv_read(p.cache, p.batch(), ko, H * D, vo, H * D + 5)
    inside = np.zeros(p.n_tokens, bool)
    inside[p.start[0]:p.start[-1]] = True
    for got, src in ((host(ko), act[:, H * D:2 * H * D]), (host(vo)[:, :H * D], act[:, 2 * H * D:3 * H * D])):
        want = R.stored(src.reshape(p.n_tokens, H, D), kind).reshape(p.n_tokens, H * D)
        assert np.array_equal(got[inside].astype(np.float64), want[inside])
        assert np.isnan(got[~inside]).all()
    # untouched bytes: everything but the new tokens' own
    units = p.page // 16
    for cache, keys in ((host(p.k), True), (host(p.v), False)):
        U = p.page_bytes // (H * units)
        mine = np.zeros((p.n_pages, H, units, U), bool)
        place = np.array([[unit_bytes(kind, D, keys, tt, d) for d in range(D)] for tt in range(16)])
        code = 16 * D * {"f16": 2, "q8_0": 1, "q4_0": 0.5}[kind]
        for s in range(len(news)):
            for pos in range(lens[s] - news[s], lens[s]):
                u = mine[p.table[s, pos // page], :, pos % page // 16]
                u[:, place[pos % 16]] = True
                if kind == "f16":
                    u[:, place[pos % 16] + 1] = True
                else:
                    for b in range(D // 32):
                        at = int(code) + (b * 16 + pos % 16) * 2
                        u[:, at:at + 2] = True
        assert (cache.reshape(mine.shape)[~mine] == 0xA5).all()


@pytest.mark.parametrize("kind", list(R.KINDS))
def test_cache_holes(kind):
    """Pages that are not there, positions before the sequence and behind the
    table: nothing is written, zeros are read."""
    H, D, page = 2, 64, 16
    p = R.Paged(kind, D, H, page, [40, 20, 30], [40, 20, 30], seed=3)
    p.table[0, 1] = -1
    p.table[1, 0] = p.n_pages
    p.lens = [40, 12, 200]                              # 8 tokens before the start; most of sequence 2 behind the table
    p.upload()
    rng = np.random.default_rng(0)
    k, v = (rng.standard_normal((p.n_tokens, H * D)).astype(np.float32) for _ in "kv")
    before = p.k.clone()
    B.mmvq_kv_write(p.cache, p.batch(), dev(k), H * D, dev(v), H * D)
    ko, vo = nan(p.n_tokens, H * D), nan(p.n_tokens, H * D)
    B.mmvq_kv_read(p.cache, p.batch(), ko, H * D, vo, H * D)
    real = np.zeros(p.n_tokens, bool)
    real[0:16] = real[32:40] = True
    for got, src in ((host(ko), k), (host(vo), v)):
        want = np.where(real[:, None], R.stored(src.reshape(-1, H, D), kind).reshape(-1, H * D), 0.0)
        assert np.array_equal(got.astype(np.float64), want)
    kept = [i for i in range(p.n_pages) if i not in (p.table[0, 0], p.table[0, 2])]
    assert np.array_equal(host(p.k)[kept], host(before)[kept])
    only = nan(p.n_tokens, H * D)
    B.mmvq_kv_read(p.cache, p.batch(), None, 0, only, H * D)
    assert np.array_equal(host(only), host(vo))


def test_cache_hints_are_hints():
    """max_new and max_len below the device's values cost nothing but time."""
    p = R.Paged("q8_0", 128, 2, 32, [70, 3], [90, 33], seed=5)
    rng = np.random.default_rng(1)
    k = rng.standard_normal((p.n_tokens, 256)).astype(np.float32)
    B.mmvq_kv_write(p.cache, p.batch(max_new=1, max_len=1), dev(k), 256, dev(k), 256)
    ko, vo = nan(p.n_tokens, 256), nan(p.n_tokens, 256)
    B.mmvq_kv_read(p.cache, p.batch(max_new=2, max_len=1), ko, 256, vo, 256)
    want = R.stored(k.reshape(-1, 2, 128), "q8_0").reshape(-1, 256)
    assert np.array_equal(host(ko).astype(np.float64), want) and np.array_equal(host(vo).astype(np.float64), want)


# --- attention -----------------------------------------------------------------------

def run_attention(p, heads, window=0, sinks=None, seed=0, qscale=1.0, max_new=None, max_len=None, ldx=0, kscale=1.0, change=None,
                  hidden=None):
    """Fills the cache, runs the operator, compares every row; returns the output."""
    import torch
    rng = np.random.default_rng(seed)
    k, v = p.fill(rng, kscale)
    if change:
        change(p, k, v)
    D, ld = p.D, heads * p.D + ldx
    q = (rng.standard_normal((p.n_tokens, ld)) * qscale).astype(np.float32)
    scale = np.float32(D ** -0.5)
    out = nan(p.n_tokens, ld)
    batch = p.batch(max_new=max_new, max_len=max_len)
    size = B.mmvq_attn_workspace(p.cache, batch, heads)
    ws = torch.full((size + 16,), 0xFF, dtype=torch.uint8, device="cuda:0")
    B.mmvq_attn(p.cache, batch, dev(q), ld, heads, float(scale), window, None if sinks is None else dev(sinks), out, ld, ws, size)
    got = host(out)
    inside = np.zeros(p.n_tokens, bool)
    for s, (new, length) in enumerate(zip(p.news, p.lens)):
        rows = slice(p.start[s], p.start[s] + new)
        inside[rows] = True
        if new == 0:
            continue
        ref, mag, smax = R.attention(q[rows, :heads * D].reshape(new, heads, D), k[s], v[s], float(scale), length - new, window, sinks,
                                     () if hidden is None else hidden[s])
        tol = R.attention_tolerance(ref, mag, smax, v[s], D)
        err = np.abs(got[rows, :heads * D].reshape(new, heads, D) - ref)
        assert (err <= tol).all(), f"sequence {s}: {(~(err <= tol)).sum()} off, worst err/tol {np.nanmax(err / tol)}"
        assert np.isnan(got[rows, heads * D:]).all()
    assert np.isnan(got[~inside]).all()
    assert (host(ws)[size:] == 0xFF).all()
    return got


@pytest.mark.parametrize("kind", list(R.KINDS))
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("H,G,news,lens,page", [
    (2, 4, [1, 1, 1], [1, 33, 700], 16),                # single tokens
    (1, 1, [1], [2050], 32),                            # one query head a key head; cut into ranges
    (2, 5, [3, 0, 5, 2], [3, 10, 300, 31], 16),         # drafted tokens, group of no power of two, an empty sequence
    (2, 2, [40, 17], [40, 97], 64),                     # chunks in the middle
    (1, 8, [150, 33], [150, 520], 128),                 # many rows
])
def test_attention(kind, D, H, G, news, lens, page):
    announce(f"attention {kind} D={D} H={H} G={G} new={news} len={lens} page={page}")
    p = R.Paged(kind, D, H, page, news, lens, seed=D + H, extra_rows=(1, 2))
    run_attention(p, H * G, seed=D, ldx=3)


@pytest.mark.parametrize("kind", list(R.KINDS))
@pytest.mark.parametrize("window", [1, 7, 32, 100, 5000])
@pytest.mark.parametrize("news,lens", [([1, 4], [600, 77]), ([90, 130], [1000, 130])])
def test_attention_window_and_sinks(kind, window, news, lens):
    announce(f"attention {kind} window={window} new={news}")
    p = R.Paged(kind, 64, 2, 32, news, lens, seed=window)
    run_attention(p, 8, window=window, seed=window)
    sinks = np.array([0.0, 2.0, -30.0, 50.0, 200.0, -np.inf, 1.0, 0.5], np.float32)
    run_attention(p, 8, window=window, sinks=sinks, seed=window)


@pytest.mark.parametrize("kind", list(R.KINDS))
@pytest.mark.parametrize("D", [128, 256])
def test_attention_window_of_wide_heads(kind, D):
    """Many rows: steps that some waves' rows see and others' do not, and a
    last tile with waves that have no rows."""
    p = R.Paged(kind, D, 1, 32, [200, 70], [500, 70], seed=D)
    run_attention(p, 1, window=40, seed=D)


@pytest.mark.parametrize("n_seqs", [2, 63, 64, 65])
def test_attention_of_many_prompts(n_seqs):
    """More workgroups than run at once, of sequences of all lengths, equal
    ones and empty ones among them."""
    rng = np.random.default_rng(n_seqs)
    news = [int(x) for x in rng.integers(70, 100, n_seqs)] if n_seqs > 2 else [1000, 70]
    news[n_seqs // 2] = 0
    lens = [new + int(x) for new, x in zip(news, rng.integers(0, 90, n_seqs) // 30 * 30)]
    p = R.Paged("q8_0", 64, 8 if n_seqs > 2 else 32, 16, news, lens, seed=n_seqs)
    run_attention(p, 8 if n_seqs > 2 else 32, seed=n_seqs)


@pytest.mark.parametrize("kind", list(R.KINDS))
@pytest.mark.parametrize("new", [3, 100])
def test_attention_hints_are_hints(kind, new):
    p = R.Paged(kind, 64, 2, 32, [new, 1], [new + 200, 900], seed=new)
    run_attention(p, 4, seed=1, max_new=1, max_len=1)


@pytest.mark.parametrize("kind", list(R.KINDS))
@pytest.mark.parametrize("new", [2, 80])
def test_attention_holes_and_rows_without_keys(kind, new):
    """Missing pages are not seen; tokens before the sequence's start and
    sequences without any page give zeros."""
    p = R.Paged(kind, 64, 2, 16, [new, new, new], [new + 50, new + 50, new + 50], seed=7)

    def change(p, k, v):
        p.table[0, 1] = -1
        p.table[1, :] = p.n_pages + 5
        p.lens[2] = new - 1                            # its first token is at position -1
        k[2], v[2] = k[2][:new - 1], v[2][:new - 1]
        p.upload()

    hidden = [range(16, 32), range(0, new + 50), ()]
    got = run_attention(p, 4, seed=2, change=change, hidden=hidden)
    assert (got[p.start[1]:p.start[2]] == 0).all() and (got[p.start[2]] == 0).all()


@pytest.mark.parametrize("window,bad_at", [(0, -2), (60, 70), (0, 40)])
@pytest.mark.parametrize("new", [4, 100])
def test_attention_infinite_values_stay_hidden(new, window, bad_at):
    """F16: an infinite value of a later token, of one behind the window of
    some rows, and of one that all rows see, reaches the rows that see it
    (whose results are infinite or NaN) and no other."""
    base = 60 if bad_at < 0 else 100                   # position of the first new token
    p = R.Paged("f16", 64, 1, 16, [new], [new + base], seed=9)
    bad = new + base + bad_at if bad_at < 0 else bad_at

    def change(p, k, v):
        rows = dev(np.full((1, 64), 1e6, np.float32))  # infinite in fp16
        start, length = dev(np.array([0, 1], np.int32)), dev(np.array([bad + 1], np.int32))
        one = B.kv_batch(start, length, p.d[2], 1, 1, 1, 1, p.wide)
        B.mmvq_kv_write(p.cache, one, dev(k[0][bad, 0].astype(np.float32)[None]), 64, rows, 64)
        v[0][bad] = 0.0                                # what the rows before must see: nothing

    import torch
    rng = np.random.default_rng(3)
    k, v = p.fill(rng)
    change(p, k, v)
    q = rng.standard_normal((new, 2 * 64)).astype(np.float32)
    out = nan(new, 128)
    batch = p.batch()
    size = B.mmvq_attn_workspace(p.cache, batch, 2)
    B.mmvq_attn(p.cache, batch, dev(q), 128, 2, 0.125, window, None, out, 128,
                torch.empty(size + 16, dtype=torch.uint8, device="cuda:0"), size)
    got = host(out).reshape(new, 2, 64)
    ref, mag, smax = R.attention(q.reshape(new, 2, 64), k[0], v[0], 0.125, base, window)
    tol = R.attention_tolerance(ref, mag, smax, v[0], 64)
    pos = base + np.arange(new)
    sees = (bad <= pos) & (bad > pos - window if window else True)
    assert sees.any()
    assert (np.abs(got - ref) <= tol)[~sees].all()
    assert not np.isfinite(got[sees]).any()


@pytest.mark.parametrize("length", [1, 40])
@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("sinks", [None, [0.5]])
def test_attention_over_infinite_keys_alone(length, new, sinks):
    """F16: rows whose every key is infinite have scores that are no numbers,
    and are not taken for rows without keys."""
    import torch
    D = 64
    p = R.Paged("f16", D, 1, 16, [new], [length + new - 1], seed=length)
    p.fill(np.random.default_rng(0))
    n = length + new - 1
    rows = dev(np.tile(np.array([1e6, -1e6], np.float32), (n, D // 2)))
    ones = dev(np.ones((n, D), np.float32))
    B.mmvq_kv_write(p.cache, p.batch(whole=True), rows, D, ones, D)
    size = B.mmvq_attn_workspace(p.cache, p.batch(), 1)
    out = torch.zeros(new, D, device="cuda:0")
    B.mmvq_attn(p.cache, p.batch(), dev(np.ones((new, D), np.float32)), D, 1, 0.125, 0,
                None if sinks is None else dev(np.array(sinks, np.float32)), out, D,
                torch.empty(size + 16, dtype=torch.uint8, device="cuda:0"), size)
    assert not np.isfinite(host(out)).any()


@pytest.mark.parametrize("new", [5, 90])
def test_attention_of_the_widest_window(new):
    """A window of 2^31 - 1 hides nothing, also where rows lie before position 0."""
    p = R.Paged("q8_0", 64, 2, 16, [new, new], [new + 20, new + 20], seed=21)

    def change(p, k, v):
        p.lens[1] = new - 3
        k[1], v[1] = k[1][:new - 3], v[1][:new - 3]
        p.upload()

    run_attention(p, 2, window=0x7fffffff, seed=22, change=change)


@pytest.mark.parametrize("kind", list(R.KINDS))
def test_attention_of_stale_slots(kind):
    """Slots that no token was written to hold NaN patterns (0xFF): never seen."""
    p = R.Paged(kind, 128, 2, 64, [1, 70], [3, 70], seed=11, fill=0xFF)
    run_attention(p, 4, seed=4)


@pytest.mark.parametrize("kind", list(R.KINDS))
@pytest.mark.parametrize("qscale,kscale", [(1e-30, 1.0), (1e12, 1e-12), (20.0, 1.0), (1.0, 1e-3), (0.01, 300.0)])
def test_attention_scales(kind, qscale, kscale):
    """Query and cache values of any size: the parts of q are scaled by its
    row's exponent, block scales of values by their token's."""
    p = R.Paged(kind, 64, 1, 32, [2, 60], [500, 60], seed=13)
    if kind == "f16" and kscale < 1e-3:                # below fp16's range
        qscale, kscale = qscale * kscale / 1e-3, 1e-3
    run_attention(p, 2, seed=5, qscale=qscale, kscale=kscale)


@pytest.mark.parametrize("kind", ["q8_0", "q4_0"])
@pytest.mark.parametrize("new", [4, 100])
def test_attention_of_uneven_scales(kind, new):
    """Value blocks whose scales differ by 2^28 between tokens and between the
    blocks of a token, subnormal and zero ones among them."""
    D, H = 128, 2
    p = R.Paged(kind, D, H, 32, [new], [new + 300], seed=31)
    rng = np.random.default_rng(31)
    n = new + 300
    raw = rng.standard_normal((n, H, D)) * np.repeat(2.0 ** rng.integers(-18, 11, (n, H, D // 32)), 32, axis=2)
    raw[5] = 0
    raw[6, :, 32:] = 0
    raw[7] *= 1e-12                                    # scales below fp16's range are 0
    raw = raw.astype(np.float32)
    kk = rng.standard_normal((n, H, D)).astype(np.float32)
    B.mmvq_kv_write(p.cache, p.batch(whole=True), dev(kk.reshape(n, -1)), H * D, dev(raw.reshape(n, -1)), H * D)

    k, v = R.stored(kk, kind), R.stored(raw, kind)
    q = (rng.standard_normal((new, 2 * H, D)) * 2).astype(np.float32)
    size = B.mmvq_attn_workspace(p.cache, p.batch(), 2 * H)
    import torch
    out = nan(new, 2 * H * D)
    B.mmvq_attn(p.cache, p.batch(), dev(q.reshape(new, -1)), 2 * H * D, 2 * H, D ** -0.5, 0, None, out, 2 * H * D,
                torch.empty(size + 16, dtype=torch.uint8, device="cuda:0"), size)
    ref, mag, smax = R.attention(q, k, v, float(np.float32(D ** -0.5)), 300)
    tol = R.attention_tolerance(ref, mag, smax, v, D)
    assert (np.abs(host(out).reshape(ref.shape) - ref) <= tol).all()


def test_offsets_past_32_bits():
    """A cache of more than 4 GiB: its last pages are written, read and attended."""
    p = R.Paged("f16", 256, 8, 1024, [3], [1030], seed=17, spare=1100)
    assert p.k.numel() > 1 << 32
    p.table[0] = [p.n_pages - 1, p.n_pages - 2]
    p.upload()
    run_attention(p, 8, seed=6)
    k, v = nan(3, 8 * 256), nan(3, 8 * 256)
    B.mmvq_kv_read(p.cache, p.batch(), k, 8 * 256, v, 8 * 256)
    assert np.isfinite(host(k)).all() and np.isfinite(host(v)).all()
    assert (host(p.k[:1090]) == 0xA5).all()


def test_rows_past_32_bits():
    """Activation rows whose strides pass 2^31 floats."""
    import torch
    ld = (1 << 30) + 4
    p = R.Paged("q8_0", 64, 1, 16, [3], [20], seed=18)
    rng = np.random.default_rng(18)
    k, v = p.fill(rng)
    q = rng.standard_normal((3, 64)).astype(np.float32)
    wide = torch.empty(2 * ld + 64, device="cuda:0")
    out = torch.empty(2 * ld + 64, device="cuda:0")
    for i in range(3):
        wide[i * ld:i * ld + 64] = dev(q[i])
    B.mmvq_attn(p.cache, p.batch(), wide, ld, 1, 0.125, 0, None, out, ld, None, 0)
    got = np.stack([host(out[i * ld:i * ld + 64]) for i in range(3)])[:, None]
    ref, mag, smax = R.attention(q[:, None], k[0], v[0], 0.125, 17)
    assert (np.abs(got - ref) <= R.attention_tolerance(ref, mag, smax, v[0], 64)).all()
    y = torch.empty(2 * ld + 64, device="cuda:0")
    B.mmvq_add_rms_norm(wide, 64, 3, ld, None, 0, None, EPS, None, 0, y, ld, None)
    _, e = R.rms_norm(q, None, None, EPS)
    got = np.stack([host(y[i * ld:i * ld + 64]) for i in range(3)])
    assert (np.abs(got - e) <= np.abs(e) * HALF32 * (1 + 1e-6)).all()


def test_nothing_to_read_is_refused():
    """Also without a tensor that would name the device."""
    p = R.Paged("f16", 64, 1, 16, [1], [1], seed=1)
    with pytest.raises(B.MMVQError):
        B.mmvq_kv_read(p.cache, p.batch(), None, 64, None, 64)


# --- verification ------------------------------------------------------------------------

def run_verify(target, kind, temp, tok, dp, start, ua, us, wide, ldt=None, ldd=None):
    import torch
    V, n, rows = target.shape[1], len(start) - 1, target.shape[0]
    ldt, ldd = ldt or V, ldd or V

    def widened(a, ld):
        b = np.full((max(1, a.shape[0]), ld), np.nan, np.float32)
        b[:a.shape[0], :V] = a
        return dev(b)

    count = torch.full((n + 1,), -7, dtype=torch.int32, device="cuda:0")
    out = torch.full((n + 1, wide), -7, dtype=torch.int32, device="cuda:0")
    size = B.mmvq_verify_workspace(n, rows, V)
    ws = torch.full((size + 16,), 0xFF, dtype=torch.uint8, device="cuda:0")
    B.mmvq_verify_draft(widened(target, ldt), ldt, V, kind, None if temp is None else dev(temp), dev(tok.astype(np.int32)),
                        None if dp is None else widened(dp, ldd), ldd, dev(np.asarray(start, np.int32)), n, rows, dev(ua), dev(us),
                        count, out, wide, ws, size)
    ec, eo = R.verify(target, kind, temp, tok, dp, start, ua, us, wide)
    gc, go = host(count), host(out)
    assert (gc[n:] == -7).all() and (go[n:] == -7).all() and (host(ws)[size:] == 0xFF).all()
    assert np.array_equal(gc[:n], ec), (gc[:n], ec)
    assert np.array_equal(go[:n], eo), (go[:n], eo)
    return ec, eo


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("V", [1, 7, 2048, 2049, 50257])
@pytest.mark.parametrize("kind", [B.TARGET_LOGITS, B.TARGET_WEIGHTS])
@pytest.mark.parametrize("drafted", [True, False])
def test_verify(V, kind, drafted):
    announce(f"verify V={V} kind={kind} drafted={drafted}")
    rng = np.random.default_rng(V * 4 + kind * 2 + drafted)
    start = np.array([0, 5, 5, 6, 14, 16])              # one sequence empty, one without drafts
    rows = start[-1]
    logits = (rng.standard_normal((rows, V)) * 3).astype(np.float32)
    q = softmax(logits + 0.5 * rng.standard_normal((rows, V)))
    tok = np.array([rng.choice(V, p=row / row.sum()) for row in q.astype(np.float64)])
    target = logits if kind == B.TARGET_LOGITS else softmax(logits)
    temp = np.array([1.0, 0.7, 0.0, 1.3, 0.5], np.float32) if kind == B.TARGET_LOGITS else None
    seen = set()
    for t in range(4):
        ua, us = rng.random(rows, np.float32), rng.random(5, np.float32)
        count, _ = run_verify(target, kind, temp if t else None, tok, q if drafted else None, start, ua, us, 8,
                              ldt=V + 3 * (t % 2), ldd=V + t % 2)
        seen.update(count.tolist())
    assert V < 3 or not drafted or len(seen) > 1        # drafts accepted and refused


def test_verify_many_sequences():
    """More sequences than a wave has lanes, rows before the first and behind the last."""
    rng = np.random.default_rng(8)
    counts = rng.integers(0, 4, 333)
    start = np.concatenate([[0], np.cumsum(counts)]) + 3
    rows, V = int(start[-1]) + 2, 300
    logits = (rng.standard_normal((rows, V)) * 2).astype(np.float32)
    q = softmax(logits + rng.standard_normal((rows, V)))
    tok = np.array([rng.choice(V, p=r / r.sum()) for r in q.astype(np.float64)])
    temp = rng.choice([0.0, 0.5, 1.0, 2.0], 333).astype(np.float32)
    run_verify(logits, B.TARGET_LOGITS, temp, tok, q, start, rng.random(rows, np.float32), rng.random(333, np.float32), 2)


@pytest.mark.parametrize("drafted", [True, False])
def test_verify_large_vocabulary(drafted):
    """More chunks of a row than a wave has lanes."""
    V, start = 300007, np.array([0, 3, 5])
    rng = np.random.default_rng(9)
    logits = (rng.standard_normal((5, V)) * 2).astype(np.float32)
    q = softmax(logits + 0.3 * rng.standard_normal((5, V)))
    tok = np.array([rng.choice(V, p=r / r.sum()) for r in q.astype(np.float64)])
    seen = set()
    for t in range(4):
        ua = rng.random(5, np.float32) * (1 if drafted else np.float32(1e-5))
        count, _ = run_verify(logits, B.TARGET_LOGITS, np.array([1.0, 0.5], np.float32), tok, q if drafted else None, start, ua,
                              rng.random(2, np.float32), 4)
        seen.update(count.tolist())
    assert len(seen) > 1


@pytest.mark.parametrize("refused", [0, 7, 8, 512, 513, 599, 600])
def test_verify_long_drafts(refused):
    """More drafted tokens than a workgroup has lanes; the first refused one anywhere."""
    V, rows = 50, 601
    rng = np.random.default_rng(refused)
    logits = rng.standard_normal((rows, V)).astype(np.float32)
    tok = logits.argmax(1)
    if refused < 600:
        tok[refused] = (tok[refused] + 1) % V
    count, out = run_verify(logits, B.TARGET_LOGITS, np.zeros(1, np.float32), tok, None, [0, rows], rng.random(rows, np.float32),
                            rng.random(1, np.float32), 700)
    assert count[0] == refused and out[0, refused] == logits[refused].argmax() and (out[0, refused + 1:] == -1).all()


def test_verify_edges():
    """Ties, masked and missing logits, tokens outside, numbers at the ends."""
    V, start = 5000, np.arange(0, 25, 2)                # one draft each
    rows, n = 24, 12
    rng = np.random.default_rng(2)
    logits = rng.standard_normal((rows, V)).astype(np.float32)
    tok = rng.integers(0, V, rows)
    temp = np.ones(n, np.float32)
    ua, us = rng.random(rows, np.float32), rng.random(n, np.float32)
    logits[0, [4000, 17]] = 50.0                        # greedy tie: the lowest index stands
    temp[0], tok[0] = 0.0, 17
    logits[2, [4000, 17]] = 50.0
    temp[1], tok[2] = -1.0, 4000
    logits[4] = -np.inf                                 # nothing is possible
    logits[6] = np.nan
    logits[8] = -np.inf                                 # all but one masked
    logits[8, 4321], tok[8], ua[8] = -3.0, 4321, 0.999
    logits[10, ::3] = np.nan
    logits[12, [5, 9]] = np.inf                         # these two share it
    tok[12], ua[12] = 9, 0.25
    tok[14], tok[16] = V, -1                            # no such tokens
    ua[18], us[9] = 0.0, 0.0
    temp[10], temp[11] = np.inf, 1e-30
    count, out = run_verify(logits, B.TARGET_LOGITS, temp, tok, None, start, ua, us, 3)
    assert out[0, 0] == 17 and count[1] == 0 and out[1, 0] == 17
    assert out[2].tolist() == [-1, -1, -1] and out[3].tolist() == [-1, -1, -1] and out[4, 0] == 4321
    run_verify(logits, B.TARGET_LOGITS, temp, tok, softmax(rng.standard_normal((rows, V))), start, ua, us, 1)
    # weights: zeros, negatives and infinities count as nothing; draft equal to target: nothing left over
    w = softmax(rng.standard_normal((rows, V)))
    w[0, :2500] = 0
    w[2, ::2] = -1
    w[4, 7] = np.inf
    w[6] = 0
    w[8] = 0
    w[8, 99] = 2.0
    ua[10], ua[8] = 1.0, 1.0                            # refused although p = q: drawn from p
    q = w.copy()
    tok[8] = 99
    run_verify(w, B.TARGET_WEIGHTS, None, tok, q, start, ua, us, 2)
    us[:] = np.float32(1 - 2.0 ** -24)
    run_verify(w, B.TARGET_WEIGHTS, None, tok, q, start, ua, us, 2)


# --- streams, graphs, together ---------------------------------------------------------------

def test_on_another_stream():
    import torch
    p = R.Paged("q8_0", 128, 2, 32, [1, 3], [400, 90], seed=1)
    rng = np.random.default_rng(6)
    p.fill(rng)
    q = dev(rng.standard_normal((4, 8 * 128)).astype(np.float32))
    batch = p.batch()
    size = B.mmvq_attn_workspace(p.cache, batch, 8)
    ws = [torch.empty(size + 16, dtype=torch.uint8, device="cuda:0") for _ in range(2)]
    a, b = nan(4, 1024), nan(4, 1024)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    B.mmvq_attn(p.cache, batch, q, 1024, 8, 0.1, 0, None, a, 1024, ws[0], size)
    B.mmvq_attn(p.cache, batch, q, 1024, 8, 0.1, 0, None, b, 1024, ws[1], size, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def decode_step(p, W, buf, st):
    """One layer's step on columns buf["x"]: norm, fused qkv product, cache,
    attention, output product, norm, language-model head, verification."""
    n, K, H, heads, D, V = st["n"], st["K"], p.H, st["heads"], p.D, st["V"]
    M = (heads + 2 * H) * D
    B.mmvq_add_rms_norm(buf["x"], K, n, K, None, 0, W["norm"], EPS, None, 0, None, 0, buf["yq"])
    B.mmvq(W["qkv"], B.Q4_K, M, K, buf["yq"], n, buf["qkv"])
    qkv = buf["qkv"]
    B.mmvq_kv_write(st["cache"], st["batch"], qkv[:, heads * D:], M, qkv[:, (heads + H) * D:], M)
    B.mmvq_attn(st["cache"], st["batch"], qkv, M, heads, D ** -0.5, 0, None, buf["att"], heads * D, buf["ws"], buf["ws"].numel())
    B.mmvq_f32(W["o"], B.Q4_K, K, heads * D, buf["att"], n, heads * D, buf["proj"])
    B.mmvq_add_rms_norm(buf["proj"], K, n, K, buf["x"], K, W["norm"], EPS, buf["h"], K, None, 0, buf["yq"])
    B.mmvq(W["head"], B.Q6_K, V, K, buf["yq"], n, buf["logits"])
    B.mmvq_verify_draft(buf["logits"], V, V, B.TARGET_LOGITS, buf["temp"], buf["tok"], None, V, p.d[0], len(p.news), n, buf["ua"],
                        buf["us"], buf["count"], buf["tokens"], st["wide"], buf["vws"], buf["vws"].numel())


@pytest.mark.parametrize("kind", list(R.KINDS))
def test_together_eager_and_captured(kind):
    """A decode step of drafted tokens through all operators, against the same
    step in 64 bits stage by stage; then captured and replayed with other
    lengths, tokens and inputs, with eager work between the replays."""
    import torch
    from quantized_decode_gemv_quantize_amd import synth
    rng = np.random.default_rng(21)
    H, heads, D, K, V = 2, 8, 64, 512, 1000
    p = R.Paged(kind, D, H, 16, [3, 1, 4], [60, 200, 33], seed=2, spare=8)
    n, M = p.n_tokens, (heads + 2 * H) * D
    st = {"n": n, "K": K, "heads": heads, "V": V, "wide": 4, "cache": p.cache, "batch": p.batch()}
    W = {"qkv": dev(synth.weights(B.Q4_K, M, K, rng)), "o": dev(synth.weights(B.Q4_K, K, heads * D, rng)),
         "head": dev(synth.weights(B.Q6_K, V, K, rng)), "norm": dev((1 + 0.1 * rng.standard_normal(K)).astype(np.float32))}
    u8 = lambda size: torch.zeros(size, dtype=torch.uint8, device="cuda:0")  # noqa: E731
    buf = {"x": nan(n, K), "yq": u8((n, K // 32 * 36)), "qkv": nan(n, M), "att": nan(n, heads * D), "proj": nan(n, K), "h": nan(n, K),
           "logits": nan(n, V), "temp": dev(np.array([0.0, 1.0, 40.0], np.float32)), "tok": dev(np.zeros(n, np.int32)),
           "ua": nan(n), "us": nan(3), "count": dev(np.zeros(3, np.int32)), "tokens": dev(np.zeros((3, 4), np.int32)),
           "ws": u8(B.mmvq_attn_workspace(st["cache"], st["batch"], heads) + 16), "vws": u8(B.mmvq_verify_workspace(3, n, V))}

    def new_inputs():
        buf["x"].copy_(dev(rng.standard_normal((n, K)).astype(np.float32)))
        buf["tok"].copy_(dev(rng.integers(0, V, n).astype(np.int32)))
        buf["ua"].copy_(dev(rng.random(n, np.float32)))
        buf["us"].copy_(dev(rng.random(3, np.float32)))

    def snapshot():
        return {k: host(buf[k]).copy() for k in ("yq", "qkv", "att", "h", "logits", "count", "tokens")}

    k, v = p.fill(rng)
    new_inputs()
    decode_step(p, W, buf, st)
    got = snapshot()
    qkv = got["qkv"].astype(np.float64)
    for s, (new, length) in enumerate(zip(p.news, p.lens)):
        rows = slice(p.start[s], p.start[s] + new)
        for c, o in ((k, heads * D), (v, (heads + H) * D)):
            c[s][length - new:] = R.stored(got["qkv"][rows, o:o + H * D].reshape(new, H, D), kind)
        ref, mag, smax = R.attention(qkv[rows, :heads * D].reshape(new, heads, D), k[s], v[s], D ** -0.5, length - new)
        tol = R.attention_tolerance(ref, mag, smax, v[s], D)
        assert (np.abs(got["att"][rows].reshape(new, heads, D) - ref) <= tol).all()
    eh, _ = R.rms_norm(host(buf["proj"]), host(buf["x"]), None, EPS)
    assert np.array_equal(got["h"].astype(np.float64), eh)
    ec, eo = R.verify(got["logits"], B.TARGET_LOGITS, host(buf["temp"]), host(buf["tok"]), None, p.start, host(buf["ua"]), host(buf["us"]), 4)
    assert np.array_equal(got["count"], ec) and np.array_equal(got["tokens"], eo)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        decode_step(p, W, buf, st)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            decode_step(p, W, buf, st)
    torch.cuda.synchronize()
    for turn in range(4):
        p.d[1].copy_(dev(np.array([60 - turn, 200 - 30 * turn, 33], np.int32)))
        new_inputs()
        graph.replay()
        torch.cuda.synchronize()
        replayed = snapshot()
        for key in ("att", "logits"):
            buf[key].fill_(float("nan"))
        decode_step(p, W, buf, st)
        eager = snapshot()
        for key in eager:
            assert np.array_equal(replayed[key], eager[key]), (turn, key)
