"""Draws by numbers between two running sums that lie close together: chunks'
sums that differ by rounding alone, small sums before a large weight."""
import numpy as np
import pytest

import draw_borders
from gpu_helpers import dev, host
from quantized_decode_gemv_quantize_amd import binding as B
from test_gpu_serve import check_sample

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(4))
def test_sample_draws_no_chunk_without_weight(seed):
    """A running sum that is larger at an entirely masked chunk than at the one before it, by rounding alone, with
    the number between the two."""
    import torch
    z, allowed = draw_borders.logits_row(seed)
    V = len(z)
    tokens, chosen = torch.full((1,), -5, dtype=torch.int32, device="cuda:0"), torch.full((1,), -5.0, device="cuda:0")
    ws = torch.full((B.mmvq_sample_workspace(1, V),), 0xA5, dtype=torch.uint8, device="cuda:0")
    B.mmvq_sample(dev(z[None]), V, V, 1, None, None, 1, dev(np.array([0.5], np.float32)), tokens, chosen, None, V, ws, ws.numel())
    got = int(host(tokens)[0])
    assert got in allowed and abs(host(chosen)[0] - np.exp(z[got].astype(np.float64)) / np.exp(z.astype(np.float64)).sum()) < 1e-6


@pytest.mark.parametrize("with_draft", [False, True])
@pytest.mark.parametrize("seed", range(4))
def test_verify_draws_no_chunk_without_weight(seed, with_draft):
    """A sequence of one row, from which the next token is drawn: one with a weight, though the running sum is
    larger at a chunk without any than at the one before it."""
    import torch
    z, allowed = draw_borders.weights_row(seed)
    V = len(z)
    count, out = (torch.full((1, n), -5, dtype=torch.int32, device="cuda:0") for n in (1, 2))
    ws = torch.full((B.mmvq_verify_workspace(1, 1, V),), 0xA5, dtype=torch.uint8, device="cuda:0")
    drafted, half = dev(np.zeros(1, np.int32)), dev(np.array([0.5], np.float32))
    B.mmvq_verify_draft(dev(z[None]), V, V, B.TARGET_WEIGHTS, None, drafted, dev(z[None]) if with_draft else None, V,
                        dev(np.array([0, 1], np.int32)), 1, 1, half, half, count, out, 2, ws, ws.numel())
    got = host(out)[0]
    assert host(count)[0, 0] == 0 and got[0] in allowed and got[1] == -1


# weights 1e-20, 1.5e-20, 1 at these places of a row, and u between the first and the first two
PLACES = [(0, 4096, 5000), (0, 8, 9), (4000, 4100, 4101), (3, 8192, 8193), (64, 512, 517), (0, 270336, 270337)]


@pytest.mark.parametrize("at", PLACES)
@pytest.mark.parametrize("kw", [dict(), dict(k=3), dict(k=8193), dict(m=1e-25)])
def test_sample_small_sums_before_a_large_weight(at, kw):
    """What lies before a chunk or a lane is not lost in that one's own sum."""
    z = np.full((1, max(at) + 1000), -np.inf, np.float32)
    z[0, list(at)] = np.log([1e-20, 1.5e-20, 1.0])
    check_sample(z, [2e-20], 1.0, **kw)
    z[0, ~np.isfinite(z[0])] = -100.0            # all others far below
    check_sample(z, [2e-20], 1.0, **kw)


@pytest.mark.parametrize("with_draft", [False, True])
@pytest.mark.parametrize("at", PLACES)
def test_verify_small_sums_before_a_large_weight(at, with_draft):
    import torch
    V = max(at) + 1000
    z = np.zeros((1, V), np.float32)
    z[0, list(at)] = [1e-20, 1.5e-20, 1.0]
    count, out = (torch.full((1, n), -5, dtype=torch.int32, device="cuda:0") for n in (1, 2))
    ws = torch.full((B.mmvq_verify_workspace(1, 1, V),), 0xA5, dtype=torch.uint8, device="cuda:0")
    u = dev(np.array([2e-20], np.float32))
    B.mmvq_verify_draft(dev(z), V, V, B.TARGET_WEIGHTS, None, dev(np.zeros(1, np.int32)), dev(z) if with_draft else None, V,
                        dev(np.array([0, 1], np.int32)), 1, 1, u, u, count, out, 2, ws, ws.numel())
    assert host(count)[0, 0] == 0 and host(out).tolist() == [[at[1], -1]]
