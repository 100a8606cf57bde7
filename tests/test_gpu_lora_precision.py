"""How far the adapters' results may lie from 64 bits, by the sums that the
launch forms: ranges of K as many as the workspace has room for, eight waves a
range that take 32 of every 256 values of K, one matrix instruction a pair of
parts and step of 32."""
import numpy as np
import pytest

from gpu_helpers import announce, dev, host
from quantized_decode_gemv_quantize_amd import binding as B
from serve_ref import U

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (B.BF16, 3), "f16": (B.F16, 6), "f32": (B.F32, 8)}   # type, instructions a step
GRID = 2.0 ** -133                             # the smallest bf16: what is below it in a value split into parts is lost
LEAST = 2.0 ** -149                            # the smallest fp32


def bound(kind, a, b, scale, x, base, splits):
    """Rows' values in 64 bits and their bounds. Parts are 8 bits each and their products exact; fp32 weights do
    without the product of the last parts (2^-28). A term of v meets 32 roundings at most inside its matrix
    instruction (a sum of 32), one at each later instruction of its wave, 7 where eight waves are joined and
    splits - 1 where the ranges are; a term of B v the 32 and the later ranks' instructions. Then the product with
    the scale and the sum with base. Sums of fp32 below 2^-126 round to LEAST."""
    instr, r, K = TYPES[kind][1], a.shape[0], a.shape[1]
    steps = -(-(-(-K // 256)) // splits)       # of 256 values, of a range
    x64, a64, b64 = x.astype(np.float64), a.astype(np.float64), b.astype(np.float64)
    v, mag = x64 @ a64.T, np.abs(x64) @ np.abs(a64).T
    n_v = 32 + instr * steps + 7 + splits - 1
    dv = U * (n_v + 2.0 ** -4) * mag + GRID * (np.abs(a64).sum(1) + np.abs(x64).sum(1, keepdims=True)) + LEAST * (K + n_v)
    y, most = v @ b64.T, (np.abs(v) + dv) @ np.abs(b64).T
    n_y = 32 + instr * -(-r // 32)
    dy = dv @ np.abs(b64).T + U * (n_y + 2.0 ** -4) * most + GRID * (np.abs(b64).sum(1) + (np.abs(v) + dv).sum(1, keepdims=True))
    dy += LEAST * (r + n_y)
    s = abs(scale)
    return base + scale * y, (s * (dy + U * most) + LEAST + U * (np.abs(base) + s * (most + dy)) + LEAST) * (1 + 1e-5)


def run(kind, K, M, r, n, scale, size=1.0, with_base=True, seed=0):
    import torch
    t = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[kind]
    rng = np.random.default_rng(seed)
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    a, b = draw(2, r, K).to(t), draw(2, M, r).to(t)
    x = (draw(n, K) * size).numpy()
    base = draw(n, M).numpy() if with_base else np.zeros((n, M), np.float32)
    ids = rng.integers(0, 2, n)
    s = B.lora_set(a.to("cuda:0"), b.to("cuda:0"), TYPES[kind][0], 2, K, M, r, None, dev(np.array([scale, scale], np.float32)))
    size_ws = B.mmvq_lora_workspace(s, n)
    out = torch.full((n, M), float("nan"), device="cuda:0")
    ws = torch.full((size_ws,), 0xFF, dtype=torch.uint8, device="cuda:0")
    B.mmvq_lora(s, dev(x), K, n, None, dev(ids.astype(np.int32)), n, dev(base), M, out, M, ws, size_ws)
    got, splits = host(out).astype(np.float64), size_ws // (4 * n * r)
    worst = 0.0
    for i in range(2):
        of = ids == i
        want, tol = bound(kind, a[i].float().numpy(), b[i].float().numpy(), scale, x[of], base[of], splits)
        if of.any():
            worst = max(worst, float((np.abs(got[of] - want) / tol).max()))
    print(f"splits {splits}, worst {worst:.3g} of the bound", flush=True)
    assert worst <= 1.0


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("K,M,r,n", [(4096, 200, 16, 1), (4096, 200, 128, 9), (14336, 130, 32, 40), (2048, 70, 256, 20), (8, 64, 8, 3),
                                     (264, 300, 40, 100), (4104, 90, 64, 1100)])
def test_lora_is_within_the_bound_of_its_sums(kind, K, M, r, n):
    announce(f"lora bound {kind} K {K} M {M} rank {r} n {n}")
    run(kind, K, M, r, n, 1.75, seed=K + n)
    run(kind, K, M, r, n, 0.5, with_base=False, seed=K + n + 1)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -110, 2.0 ** -120, 2.0 ** -126, 2.0 ** -135])
def test_lora_of_tiny_values(kind, size):
    """Down to the smallest numbers: what a value has below 2^-133 may be lost, and nothing else."""
    run(kind, 512, 60, 16, 5, 1.0, size, with_base=False, seed=7)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("K,r,n", [(64, 8, 3), (4096, 16, 5), (1000, 72, 70), (264, 256, 20), (4096, 32, 1100)])
def test_lora_loses_no_part_of_a_value(kind, K, r, n):
    """One term a sum, so that nothing rounds: activations times 1, the first matrix's weights times 1 and the second
    one's come out with all their bits."""
    import torch
    announce(f"lora parts {kind} K {K} rank {r} n {n}")
    t = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[kind]
    M = 130
    rng = np.random.default_rng(K + r)
    full = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    place, rank_of = rng.integers(0, K, n), rng.integers(0, r, M)
    one_rank = torch.zeros(1, M, r)
    one_rank[0, np.arange(M), rank_of] = 1.0
    value = full(n)
    hot = torch.zeros(n, K)
    hot[np.arange(n), place] = 1.0
    first = torch.zeros(1, r, K)
    first[0, 0] = 1.0

    def out(x, a, b):
        s = B.lora_set(a.to(t).to("cuda:0"), b.to(t).to("cuda:0"), TYPES[kind][0], 1, K, M, r)
        got = torch.full((n, M), float("nan"), device="cuda:0")
        ws = torch.full((B.mmvq_lora_workspace(s, n),), 0xFF, dtype=torch.uint8, device="cuda:0")
        B.mmvq_lora(s, x.to("cuda:0"), K, n, None, torch.zeros(n, dtype=torch.int32, device="cuda:0"), n, torch.zeros(n, M, device="cuda:0"),
                    M, got, M, ws, ws.numel())
        return got.cpu()

    assert torch.equal(out(hot * value[:, None], torch.ones(1, r, K), one_rank), value[:, None].expand(n, M))
    a = full(1, r, K)
    assert torch.equal(out(hot, a, one_rank), a.to(t).float()[0][rank_of][:, place].t())
    b = full(1, M, r)
    assert torch.equal(out(hot, first, b), b.to(t).float()[0, :, 0].expand(n, M))
