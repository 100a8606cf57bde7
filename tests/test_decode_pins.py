"""The bounds of tests/decode_pins.py on the CPU: the bits that the attention
operator states keep them, five fewer of either part do not."""
import numpy as np
import pytest

import decode_pins as P
import decode_ref as R


@pytest.mark.parametrize("kind", list(R.KINDS))
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("new", [3, 8, 12, 40])
@pytest.mark.parametrize("part", ["q", "weights"])
def test_fewer_bits_are_seen(kind, D, new, part):
    k, v, q = P.inputs(kind, D, part, new)
    k, v = R.stored(k, kind), R.stored(v, kind)
    scale = float(np.float32(D ** -0.5))
    ref, mag = P.reference(q, k, v, scale)
    tol = P.tolerance(mag, part, v)
    assert np.abs(ref).max() > 0

    def off(q_bits, w_bits):
        return (np.abs(P.model(q, k, v, scale, q_bits, w_bits) - ref) / tol).max()

    assert off(53, 53) < 1e-3
    assert off(22, 21) < 1
    assert off(16, 53) > 1.5 if part == "q" else off(53, 16) > 1.5
