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
