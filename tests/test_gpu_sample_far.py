"""Sampling where the kept tokens' weights lie far apart."""
import numpy as np
import pytest

from gpu_helpers import announce
from test_gpu_serve import check_sample

pytestmark = pytest.mark.gpu


def far_row(V, counts, tops, rng):
    """Per chunk of 4096 logits some finite ones, from its top down to 2 below; all others masked."""
    z = np.full(V, -np.inf, np.float32)
    for c, (n, top) in enumerate(zip(counts, tops)):
        size = min(4096, V - 4096 * c)
        z[4096 * c + rng.choice(size, n, replace=False)] = top - 2 * rng.random(n) * (np.arange(n) > 0)
    return z


@pytest.mark.parametrize("counts", [(1, 20), (30, 25, 5), (60, 150), (250, 240), (256, 256, 256), (20, 0, 200, 100)])
@pytest.mark.parametrize("fall", [14.0, 20.0, 30.0])
def test_sample_chunks_far_below_the_top(counts, fall):
    """Strictly masked rows: a chunk's largest weight is e^-46 to e^-100 of the row's, more than 255 quarter octaves
    down, and its tokens are kept all the same where the filters say so."""
    announce(f"far chunks {counts} fall {fall}")
    rng = np.random.default_rng(int(sum(counts) * fall))
    T, n, near = 0.3, sum(counts), counts[0]
    V = 4096 * (len(counts) - 1) + 3500
    tops = [20.0] + [20.0 - fall - 0.1 * c for c in range(1, len(counts))]
    k = [n + 9, n, near + (n - near) // 2, near + 1, near, 0, 0, n - 1, 0]
    p = [1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0 - 2.0 ** -24, 1.0 - 2.0 ** -24]
    m = [0.0, 0.0, 0.0, 0.0, 0.0, 1e-30, 1e-38, 0.0, 0.0]
    z = np.stack([far_row(V, counts, tops, rng) for _ in k])
    for u in (rng.random(len(k)), np.full(len(k), 1 - 2.0 ** -24)):
        check_sample(z, u, T, k, p, m)
