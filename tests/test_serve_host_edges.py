"""Calls of the operators of a step over many requests at the edges of what
they take, without a GPU: no rows, for which buffers may be NULL whatever their
strides, and many requests."""
import pytest

from quantized_decode_gemv_quantize_amd import binding as B


@pytest.mark.parametrize("ldb,ldo", [(50, 50), (50, 52), (60, 50)])
def test_lora_of_no_rows_takes_any_strides(ldb, ldo):
    """Without rows base and out may both be NULL, which does not make them one buffer."""
    s = B.lora_set(None, None, B.F16, 3, 64, 50, 16)
    assert B.lib().mmvq_lora(s, None, 64, 0, None, None, 0, None, ldb, None, ldo, None, 0, None) == 0


@pytest.mark.parametrize("ldl,ldp", [(100, 100), (100, 120), (120, 100)])
def test_sample_of_no_rows_takes_any_strides(ldl, ldp):
    assert B.lib().mmvq_sample(None, ldl, 100, 0, None, None, 0, None, None, None, None, ldp, None, 0, None) == 0


@pytest.mark.parametrize("n_seqs", [(1 << 20) + 1, (1 << 31) - 1])
def test_lora_and_sample_of_any_number_of_requests(n_seqs):
    """The number of requests bounds the arrays that rows name places in; no launch depends on it."""
    s = B.lora_set(None, None, B.F16, 3, 64, 50, 16)
    assert B.lib().mmvq_lora(s, None, 64, 0, None, 1 << 20, n_seqs, None, 50, None, 50, None, 0, None) == 0
    assert B.lib().mmvq_sample(None, 100, 100, 0, None, None, n_seqs, None, None, None, None, 100, None, 0, None) == 0
