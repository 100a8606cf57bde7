"""Operators between the mat-vecs on the GPU, at the edges of what their
header allows."""
import numpy as np
import pytest

import decode_ref as R
from gpu_helpers import announce, dev, host
from quantized_decode_gemv_quantize_amd import binding as B

pytestmark = pytest.mark.gpu


def floats(*shape):
    import torch
    return torch.full(shape, float("nan"), device="cuda:0")


def ints(*shape):
    import torch
    return torch.full(shape, -7, dtype=torch.int32, device="cuda:0")


def space(size):
    import torch
    return torch.empty(size, dtype=torch.uint8, device="cuda:0")


# --- nothing to do ----------------------------------------------------------------------

def test_empty_tensors():
    """No columns, tokens, sequences or rows: tensors without an element."""
    p = R.Paged("q8_0", 64, 2, 16, [1], [20], seed=1)
    before = p.k.clone()
    for n_seqs in (0, 1):
        start = dev(np.zeros(n_seqs + 1, np.int32))
        batch = B.kv_batch(start, p.d[1][:n_seqs], p.d[2][:n_seqs], n_seqs, 0, 1, 20, p.wide)
        B.mmvq_kv_write(p.cache, batch, floats(0, 128), 128, floats(0, 128), 128)
        B.mmvq_kv_read(p.cache, batch, floats(0, 128), 128, floats(0, 128), 128)
        size = B.mmvq_attn_workspace(p.cache, batch, 4)
        assert size == 0
        B.mmvq_attn(p.cache, batch, floats(0, 256), 256, 4, 0.1, 0, None, floats(0, 256), 256, space(0), size)
    assert np.array_equal(host(p.k), host(before))
    B.mmvq_add_rms_norm(floats(0, 64), 64, 0, 64, floats(0, 64), 64, floats(64), 1e-5, floats(0, 64), 64, floats(0, 64), 64, space(0))
    B.mmvq_dequantize_q8_1(space(0), 64, 0, floats(0, 64), 64)
    size = B.mmvq_verify_workspace(0, 0, 100)
    B.mmvq_verify_draft(floats(0, 100), 100, 100, B.TARGET_LOGITS, floats(0), ints(0), floats(0, 100), 100, ints(1), 0, 0,
                        floats(0), floats(0), ints(0), ints(0, 3), 3, space(size), size)


@pytest.mark.parametrize("drafted", [True, False])
def test_sequences_without_any_row(drafted):
    """Each gets 0 and -1."""
    size = B.mmvq_verify_workspace(3, 0, 100)
    count, tokens = ints(3), ints(3, 2)
    B.mmvq_verify_draft(floats(0, 100), 100, 100, B.TARGET_LOGITS, None, ints(0), floats(1, 100) if drafted else None, 100,
                        dev(np.zeros(4, np.int32)), 3, 0, floats(0), dev(np.full(3, 0.5, np.float32)), count, tokens, 2,
                        space(size), size)
    assert host(count).tolist() == [0, 0, 0] and (host(tokens) == -1).all()


def test_on_the_default_stream_as_an_object():
    import torch
    x, y = dev(np.ones((2, 64), np.float32)), floats(2, 64)
    B.mmvq_add_rms_norm(x, 64, 2, 64, None, 0, None, 0.0, None, 0, y, 64, None, stream=torch.cuda.default_stream())
    assert (host(y) == 1).all()


# --- sinks of any size ------------------------------------------------------------------

@pytest.mark.parametrize("kind", list(R.KINDS))
@pytest.mark.parametrize("new,length", [(1, 40), (1, 3000), (90, 130)])
def test_sinks_to_the_ends_of_fp32(kind, new, length):
    """A sink far above all scores leaves nothing for the keys, one far below
    them takes nothing; in one launch, with a join, and of many rows."""
    announce(f"sinks {kind} new={new} len={length}")
    top = float(np.finfo(np.float32).max)
    sinks = np.array([top, 3e38, 2e38, 1.0, -2e38, -3e38, -top, -np.inf], np.float32)
    p = R.Paged(kind, 64, 1, 32, [new], [length], seed=3)
    rng = np.random.default_rng(length)
    k, v = p.fill(rng)
    q = rng.standard_normal((new, 8, 64)).astype(np.float32)
    batch = p.batch()
    size = B.mmvq_attn_workspace(p.cache, batch, 8)
    out = floats(new, 512)
    B.mmvq_attn(p.cache, batch, dev(q.reshape(new, 512)), 512, 8, 0.125, 0, dev(sinks), out, 512, space(size + 16), size)
    got = host(out).reshape(new, 8, 64)
    ref, mag, smax = R.attention(q, k[0], v[0], 0.125, length - new, 0, sinks.astype(np.float64))
    assert (np.abs(got - ref) <= R.attention_tolerance(ref, mag, smax, v[0], 64)).all()
    assert (got[:, :3] == 0).all() and np.abs(got[:, 3:]).max() > 0.01


# --- little left beside a refused token ---------------------------------------------------

def verify(target, kind, temp, tok, start, ua, us, wide):
    V, n, rows = target.shape[1], len(start) - 1, len(target)
    size = B.mmvq_verify_workspace(n, rows, V)
    count, out = ints(n), ints(n, wide)
    B.mmvq_verify_draft(dev(target), V, V, kind, None if temp is None else dev(temp), dev(tok.astype(np.int32)), None, V,
                        dev(np.asarray(start, np.int32)), n, rows, dev(ua), dev(us), count, out, wide, space(size), size)
    ec, eo = R.verify(target, kind, temp, tok, None, start, ua, us, wide)
    gc, go = host(count), host(out)
    assert np.array_equal(gc, ec) and np.array_equal(go, eo), (gc, ec, go, eo)
    return gc, go


@pytest.mark.parametrize("kind", [B.TARGET_LOGITS, B.TARGET_WEIGHTS])
@pytest.mark.parametrize("V", [1000, 9001, 300007])
@pytest.mark.parametrize("x", [0, 3, 400, 999])
def test_refused_token_with_nearly_all_of_its_chunk(kind, V, x):
    """Without draft probabilities: what is left of the refused token's chunk
    is a millionth of it, or 10^-20 beside weights in other chunks, where the
    chunk's sum less the token's weight would be nothing or noise. Numbers of 0
    draw the lowest index that has a weight."""
    announce(f"refused kind={kind} V={V} x={x}")
    rng = np.random.default_rng(V + x)
    us = np.array([0.0, 0.0, 0.25, 0.5, 0.999, 0.0, 0.6], np.float32)
    n = len(us)
    w = rng.random((2 * n, V)) + 0.5                    # weights of each sequence's two rows
    for s in range(n):
        row = w[2 * s]
        first = slice(0, 1000)                          # inside the first chunk, where x is
        if s % 2 == 0 or V == 1000:
            row *= 3e-6 / row.sum()                     # all the rest: a few millionths
        else:
            row[first] *= 1e-20
            row[1000:5000] *= 1e-20                     # to the chunk's end and a little further
            row[5000:] *= 0.02 / row[5000:].sum()
        row[x] = 1.0
    ua = np.full(2 * n, np.float32(1 - 2.0 ** -24))
    tok = np.full(2 * n, x)
    with np.errstate(divide="ignore"):
        target = (np.log(w) if kind == B.TARGET_LOGITS else w).astype(np.float32)
    count, out = verify(target, kind, None, tok, np.arange(0, 2 * n + 1, 2), ua, us, 2)
    assert (count == 0).all() and (out[:, 0] != x).all()
    low = 1 if x == 0 else 0
    assert (out[us == 0, 0] == low).all()


# --- batches of unlike sequences ----------------------------------------------------------

@pytest.mark.parametrize("kind", list(R.KINDS))
@pytest.mark.parametrize("D,H,G,news,lens", [
    (128, 2, 4, [200] + [1] * 7, [260, 700, 33, 1, 512, 90, 301, 16]),      # a prompt's chunk beside single tokens
    (64, 1, 8, [1] * 5 + [7, 2, 1, 3], [2600, 40, 1, 17, 300, 7, 90, 64, 3]),   # a long sequence among short ones, drafts beside
    (256, 2, 2, [1, 90, 5, 0], [900, 90, 40, 55]),
])
@pytest.mark.parametrize("window", [0, 50])
def test_attention_of_unlike_sequences(kind, D, H, G, news, lens, window):
    """Every form of a launch works on all sequences; one call, and the same
    sequences in two calls, the long chunks apart from the rest."""
    announce(f"unlike {kind} D={D} new={news} len={lens} window={window}")
    p = R.Paged(kind, D, H, 32, news, lens, seed=D)
    rng = np.random.default_rng(D + window)
    k, v = p.fill(rng)
    heads, n = H * G, p.n_tokens
    q = rng.standard_normal((n, heads, D)).astype(np.float32)
    qd, scale = dev(q.reshape(n, -1)), float(np.float32(D ** -0.5))

    def run(batch, out):
        size = B.mmvq_attn_workspace(p.cache, batch, heads)
        B.mmvq_attn(p.cache, batch, qd, heads * D, heads, scale, window, None, out, heads * D, space(size + 16), size)

    def check(out, seqs):
        got = host(out).reshape(n, heads, D)
        for s in range(len(news)):
            rows = slice(p.start[s], p.start[s] + news[s])
            if s not in seqs:
                assert np.isnan(got[rows]).all()
            elif news[s]:
                ref, mag, smax = R.attention(q[rows], k[s], v[s], scale, lens[s] - news[s], window)
                tol = R.attention_tolerance(ref, mag, smax, v[s], D)
                assert (np.abs(got[rows] - ref) <= tol).all(), s

    whole = floats(n, heads * D)
    run(p.batch(), whole)
    check(whole, range(len(news)))
    # parts of the batch by descriptors of their own: sequences a .. b-1
    long = int(np.argmax(news))
    for a, b in ((long, long + 1), (long + 1, len(news)), (0, long)):
        if a == b or max(news[a:b]) == 0:
            continue
        part = B.kv_batch(p.d[0][a:b + 1], p.d[1][a:b], p.d[2][a:b], b - a, n, max(news[a:b]), max(lens[a:b]), p.wide, p.wide)
        out = floats(n, heads * D)
        run(part, out)
        check(out, range(a, b))
