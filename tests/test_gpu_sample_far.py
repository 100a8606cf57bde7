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


def peaks_over_floor(V, depth, rng):
    """Logits of a few likely tokens in the second half over a broad floor `depth` below."""
    z = (rng.standard_normal(V) * 0.5 - depth).astype(np.float32)
    z[rng.integers(V // 2, V, 5)] = rng.standard_normal(5)
    return z


SMALLEST = np.array([0.0, 1e-38, 1e-30, 1e-18, 2.0 ** -40, 2.0 ** -24, 0.25], np.float32)


@pytest.mark.parametrize("n", [300, 2000, 5000])
@pytest.mark.parametrize("depth", [20.0, 36.0, 60.0])
def test_sample_small_numbers_among_listed_tokens(n, depth):
    """The first token whose running sum passes u * total, also where that and all weights before it are far below
    2^-50 of the largest; u = 0 draws the first kept token."""
    announce(f"small numbers, {n} tokens, depth {depth}")
    rng = np.random.default_rng(n + int(depth))
    z = np.full((len(SMALLEST), 9000), -np.inf, np.float32)
    for row in z:
        at = np.sort(rng.choice(9000, n, replace=False))
        row[at] = peaks_over_floor(n, depth, rng)
    check_sample(z, SMALLEST, 1.0, [n + 1] * len(SMALLEST))
    check_sample(z, SMALLEST, 1.0, n - n // 7)


@pytest.mark.parametrize("V,depth", [(9000, 200.0), (20000, 60.0), (20000, 90.0), (20000, 700.0)])
def test_sample_small_numbers_among_many_tokens(V, depth):
    """The same with the border among more tokens than are listed, all of them in the last bin of the weight: a
    chunk of the row that holds nothing else is drawn from by u = 0."""
    announce(f"small numbers, V {V}, depth {depth}")
    rng = np.random.default_rng(V + int(depth))
    z = np.stack([peaks_over_floor(V, depth, rng) for _ in SMALLEST])
    for k in (2000, V - V // 7, V - 1):
        check_sample(z, SMALLEST, 1.0, k)
    check_sample(z, SMALLEST, 1.0, V - 1, 1.0, 1e-30)
