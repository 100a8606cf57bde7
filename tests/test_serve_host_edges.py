"""Calls of the operators of a step over many requests that hold nothing,
without a GPU: buffers may be NULL then, whatever their strides."""
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
