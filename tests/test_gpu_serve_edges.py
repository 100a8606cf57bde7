"""Calls of the operators of a step over many requests at the edges of what
their documentation allows: the most rows and requests, no requests at all,
outputs that are not wanted, NaN of every kind, one workspace for two calls in
turn, and one state for two calls in one graph."""
import numpy as np
import pytest

import serve_ref as R
from gpu_helpers import announce, dev, host
from quantized_decode_gemv_quantize_amd import binding as B

pytestmark = pytest.mark.gpu


def nan(*shape):
    import torch
    return torch.full(shape, float("nan"), device="cuda:0")


def ints(*shape, value=77, dtype=None):
    import torch
    return torch.full(shape, value, dtype=dtype or torch.int32, device="cuda:0")


def garbage(n):
    import torch
    return torch.full((max(n, 1),), 0xA5, dtype=torch.uint8, device="cuda:0")


def settings(T=None, k=None, p=None, m=None):
    arr = lambda v, t: None if v is None else dev(np.asarray(v, dtype=t))
    return B.sampling(arr(T, np.float32), arr(k, np.int32), arr(p, np.float32), arr(m, np.float32))


def test_pages_of_the_most_requests():
    """2^20 requests of one token each, one page a request, given and taken back."""
    import torch
    n = 1 << 20
    rng = np.random.default_rng(0)
    free = rng.permutation(n).astype(np.int32)
    table, held, fd, n_free = ints(n, 1), ints(n, value=0), dev(free), dev(np.array([n], np.int32))
    pool = B.kv_pool(table, held, fd, n_free, 1, n, 16, 1)
    ws = garbage(B.mmvq_kv_plan_workspace(n))
    start, length, seq, pos, slot, missing = ints(n + 1), ints(n), ints(n), ints(n), ints(n, dtype=torch.int64), ints(1)
    announce("plan of 2^20 requests")
    B.mmvq_kv_plan(pool, ints(n, value=0), ints(n, value=1), n, n, start, length, seq, pos, slot, missing, ws, ws.numel())
    at = np.arange(n)
    assert np.array_equal(host(start), np.arange(n + 1)) and (host(length) == 1).all() and np.array_equal(host(seq), at)
    assert (host(pos) == 0).all() and np.array_equal(host(slot), free.astype(np.int64) * 16)
    assert np.array_equal(host(table)[:, 0], free) and (host(held) == 1).all() and host(n_free)[0] == 0 and host(missing)[0] == 0
    announce("release of 2^20 requests")
    B.mmvq_kv_release(pool, n, ints(n, value=0))
    assert host(n_free)[0] == n and np.array_equal(host(fd), free) and (host(table) == -1).all() and (host(held) == 0).all()


def test_lora_of_the_most_rows():
    """2^20 rows: runs of rows of an adapter, single ones, and rows of none."""
    import torch
    n, K, M, r, count = 1 << 20, 8, 3, 8, 5
    gen = torch.Generator().manual_seed(1)
    a = torch.randn(count, r, K, generator=gen).bfloat16().to("cuda:0")
    b = torch.randn(count, M, r, generator=gen).bfloat16().to("cuda:0")
    s = B.lora_set(a, b, B.BF16, count, K, M, r)
    x, base = torch.randn(n, K, generator=gen).to("cuda:0"), torch.randn(n, M, generator=gen).to("cuda:0")
    row = torch.arange(n, device="cuda:0")
    ids = torch.where(row % 1000 < 500, row // 1000 % count, row % 7 - 1).int()
    out, ws = nan(n, M), garbage(B.mmvq_lora_workspace(s, n))
    announce("lora of 2^20 rows")
    B.mmvq_lora(s, x, K, n, None, ids, n, base, M, out, M, ws, ws.numel())
    got, dt = out.double(), torch.float64
    real = (ids >= 0) & (ids < count)
    j = torch.where(real, ids, 0).long()
    v = (a.to(dt)[j] * x.to(dt)[:, None, :]).sum(-1)
    va = (a.to(dt)[j] * x.to(dt)[:, None, :]).abs().sum(-1)
    want = base.to(dt) + torch.where(real[:, None], (b.to(dt)[j] * v[:, None, :]).sum(-1), 0.0)
    # sums of 8 products of three parts, twice, each term off by some 2^-24 of it: 2 * 3 * 8 roundings and the last sum's
    tol = 64 * 2.0 ** -24 * (base.to(dt).abs() + (b.to(dt).abs()[j] * va[:, None, :]).sum(-1))
    assert bool(((got - want).abs() <= tol).all())
    assert torch.equal(out[~real], base[~real])


def test_lora_without_requests():
    """No request at all: every row gets its base, and there is no adapter array."""
    import torch
    a, b = torch.ones(1, 8, 64, device="cuda:0"), torch.ones(1, 70, 8, device="cuda:0")
    s = B.lora_set(a, b, B.F32, 1, 64, 70, 8)
    base, out = torch.randn(5, 70, device="cuda:0"), nan(5, 70)
    ws = garbage(B.mmvq_lora_workspace(s, 5))
    B.mmvq_lora(s, torch.ones(5, 64, device="cuda:0"), 64, 5, ints(5, value=0), None, 0, base, 70, out, 70, ws, ws.numel())
    assert torch.equal(out, base)


def test_lora_adapters_and_projections_in_turn():
    """Two calls in place on one output, as for two adapters of a request, with one workspace; the second sees the first."""
    import torch
    K, M, n = 256, 300, 9
    rng = np.random.default_rng(3)
    w = lambda *s: dev(rng.standard_normal(s).astype(np.float32))
    a, b = w(4, 16, K), w(4, M, 16)
    s = B.lora_set(a, b, B.F32, 4, K, M, 16)
    x, base = w(n, K), w(n, M)
    one, two = dev(rng.integers(0, 4, n).astype(np.int32)), dev(rng.integers(-1, 4, n).astype(np.int32))
    ws = garbage(B.mmvq_lora_workspace(s, n))
    out = base.clone()
    for ids in (one, two):
        B.mmvq_lora(s, x, K, n, None, ids, n, out, M, out, M, ws, ws.numel())
    apart = base
    for ids in (one, two):
        fresh, w2 = nan(n, M), garbage(B.mmvq_lora_workspace(s, n))
        B.mmvq_lora(s, x, K, n, None, ids, n, apart, M, fresh, M, w2, w2.numel())
        apart = fresh
    assert torch.equal(out, apart)


@pytest.mark.parametrize("n", [32767, 32768, 32769, 70000])
def test_sample_many_rows(n):
    """More rows than one dimension of a launch: each row is its own, in all outputs."""
    announce(f"sample {n} rows")
    V, kinds = 5, 97
    rng = np.random.default_rng(n)
    z = (rng.standard_normal((kinds, V)) * 2).astype(np.float32)
    T, k = rng.choice([0.0, 0.5, 1.0, 2.0], kinds).astype(np.float32), rng.integers(0, 6, kinds)
    p, m = rng.choice([0.4, 0.8, 1.0], kinds).astype(np.float32), rng.choice([0.0, 0.1], kinds).astype(np.float32)
    u = rng.random(kinds).astype(np.float32)
    of = np.arange(n) % kinds
    import torch
    tokens, chosen, probs = ints(n), nan(n), nan(n, V)
    ws = garbage(B.mmvq_sample_workspace(n, V))
    B.mmvq_sample(dev(z[of]), V, V, n, settings(T, k, p, m), dev(of.astype(np.int32)), kinds, dev(u[of]), tokens, chosen, probs, V, ws, ws.numel())
    w = np.stack([R.distribution(z[i], T[i], k[i], p[i], m[i]) for i in range(kinds)])
    w /= w.sum(1, keepdims=True)
    drawn = np.array([R.drawn(w[i], u[i]) for i in range(kinds)])
    assert np.array_equal(host(tokens), drawn[of])
    assert (np.abs(host(probs) - w[of]) <= w[of] * R.U * (1 + 1e-4) + 2.0 ** -150).all()
    assert (np.abs(host(chosen) - w[np.arange(kinds), drawn][of]) <= R.U * (1 + 1e-4)).all()


def test_sample_outputs_that_are_not_wanted():
    """Each output alone; without tokens and their probabilities no numbers are read."""
    import torch
    rng = np.random.default_rng(4)
    n, V = 6, 9000
    z, u = dev((rng.standard_normal((n, V)) * 3).astype(np.float32)), dev(rng.random(n).astype(np.float32))
    params = settings([1.0, 0.0, 0.7, 1.0, 1.0, 2.0], [0, 0, 40, 5000, 0, 0], [1.0, 1.0, 0.9, 0.99, 0.5, 1.0], [0.0, 0.0, 0.0, 0.0, 0.0, 0.2])
    ws = garbage(B.mmvq_sample_workspace(n, V))
    run = lambda u, t, c, p: B.mmvq_sample(z, V, V, n, params, None, n, u, t, c, p, V, ws, ws.numel())
    tokens, chosen, probs = ints(n), nan(n), nan(n, V)
    run(u, tokens, chosen, probs)
    t, c, p = ints(n), nan(n), nan(n, V)
    run(u, t, None, None)
    run(u, None, c, None)
    run(None, None, None, p)
    assert torch.equal(t, tokens) and torch.equal(c, chosen) and torch.equal(p, probs)


def test_sample_without_requests():
    """No request: token -1, chosen and probs 0, whatever the rows hold."""
    z = dev(np.array([[1.0, np.inf, np.nan], [0.0, 1.0, 2.0]], np.float32))
    for params in (None, settings(None, None, None, None)):
        tokens, chosen, probs = ints(2), nan(2), nan(2, 3)
        ws = garbage(B.mmvq_sample_workspace(2, 3))
        B.mmvq_sample(z, 3, 3, 2, params, ints(2, value=0), 0, dev(np.zeros(2, np.float32)), tokens, chosen, probs, 3, ws, ws.numel())
        assert (host(tokens) == -1).all() and (host(chosen) == 0).all() and (host(probs) == 0).all()


@pytest.mark.parametrize("bits", [0x7F800001, 0x7FC00000, 0xFF800001, 0xFFFFFFFF])
@pytest.mark.parametrize("V", [70, 5000, 12289])
def test_sample_every_kind_of_nan(bits, V):
    """Quiet and signalling NaN of either sign weigh nothing, in filtered, plain and greedy rows, listed or not."""
    import torch
    rng = np.random.default_rng(V)
    z = (rng.standard_normal((6, V)) * 2).astype(np.float32)
    holes = rng.random((6, V)) < 0.3
    clean = np.where(holes, -np.inf, z).astype(np.float32)
    raw = np.where(holes, np.uint32(bits), z.view(np.uint32))
    params = settings([1.0, 0.0, 1.0, 0.8, 1.0, 9.0], [0, 0, 20, 0, 0, V - 1], [1.0, 1.0, 1.0, 0.9, 1.0, 0.999], [0.0, 0.0, 0.0, 0.0, 0.2, 0.0])
    u = dev(rng.random(6).astype(np.float32))
    got = []
    for logits in (dev(raw.view(np.int32)).view(torch.float32), dev(clean)):
        tokens, chosen, probs = ints(6), nan(6), nan(6, V)
        ws = garbage(B.mmvq_sample_workspace(6, V))
        B.mmvq_sample(logits, V, V, 6, params, None, 6, u, tokens, chosen, probs, V, ws, ws.numel())
        got.append((host(tokens), host(chosen), host(probs)))
    for a, b in zip(*got):
        assert np.array_equal(a, b)
    assert (got[0][2][holes] == 0).all()


def test_two_steps_in_one_graph():
    """A graph of two steps of the same pool, the second from the first one's lengths: replayed, the pool's state goes on."""
    import torch
    rng = np.random.default_rng(9)
    n, n_rows = 20, 60
    pool = R.Pool(n, 12, 200, 16, 200, rng)
    table, held, free, n_free = dev(pool.table), dev(pool.held), dev(pool.free), dev(np.array([pool.n_free], np.int32))
    handle = B.kv_pool(table, held, free, n_free, pool.wide, pool.n_pages, pool.page, pool.wide)
    ws = garbage(B.mmvq_kv_plan_workspace(n))
    cached, new, start, slot = ints(n, value=0), ints(n, value=0), [ints(n + 1) for _ in range(2)], [ints(n_rows, dtype=torch.int64) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(2):
            B.mmvq_kv_plan(handle, cached, new, n, n_rows, start[i], cached, None, None, slot[i], None, ws, ws.numel())
    at = np.zeros(n, np.int64)
    cached.zero_()
    for step in range(4):
        fresh = rng.integers(0, 4, n)
        new.copy_(dev(fresh.astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            want = pool.plan(at, fresh, n_rows)
            assert np.array_equal(host(start[i]), want[0]) and np.array_equal(host(slot[i]), want[4])
            at = want[1].astype(np.int64)
        assert np.array_equal(host(cached), at) and np.array_equal(host(table), pool.table) and host(n_free)[0] == pool.n_free


@pytest.mark.parametrize("kind", [B.F32, B.F16, B.BF16])
def test_embed_rows_beyond_the_caches(kind):
    """More than 32 MB of rows, of an odd length and with a gap between them."""
    import torch
    n, K, vocab, ldo = 9001, 1001, 50, 1006
    t = {B.F32: torch.float32, B.F16: torch.float16, B.BF16: torch.bfloat16}[kind]
    table = torch.randn(vocab, K, generator=torch.Generator().manual_seed(2)).to(t).to("cuda:0")
    ids = torch.arange(n, device="cuda:0", dtype=torch.int32) * 7 % (vocab + 1) - 1
    out = nan(n, ldo)
    announce(f"embed {n} rows of {K}")
    B.mmvq_embed(table, kind, vocab, K, ids, n, 0.75, out, ldo)
    want = torch.where((ids >= 0)[:, None], table.float()[ids.clamp(min=0).long()] * 0.75, 0.0)
    assert torch.equal(out[:, :K], want) and bool(out[:, K:].isnan().all())


@pytest.mark.parametrize("kind,r", [(B.BF16, 16), (B.F16, 32), (B.F32, 64)])
def test_lora_rows_beyond_the_caches(kind, r):
    """More than 32 MB of x and of out, odd M, gaps between rows, in place and not."""
    import torch
    n, K, M, count = 2100, 4104, 4099, 3
    t = {B.F32: torch.float32, B.F16: torch.float16, B.BF16: torch.bfloat16}[kind]
    gen = torch.Generator().manual_seed(r)
    a = (torch.randn(count, r, K, generator=gen) / 64).to(t).to("cuda:0")
    b = torch.randn(count, M, r, generator=gen).to(t).to("cuda:0")
    s = B.lora_set(a, b, kind, count, K, M, r)
    x, base = torch.randn(n, K + 4, generator=gen).to("cuda:0"), torch.randn(n, M + 1, generator=gen).to("cuda:0")
    ids = (torch.arange(n, device="cuda:0") // 700).int()
    ids[5::97] = -1
    dt, xs = torch.float64, x[:, :K].double()
    want, size = base[:, :M].double(), base[:, :M].double().abs()
    for i in range(count):
        of = ids == i
        v, va = xs[of] @ a[i].to(dt).t().contiguous(), xs[of].abs() @ a[i].to(dt).abs().t().contiguous()
        want[of] += v @ b[i].to(dt).t().contiguous()
        size[of] += va @ b[i].to(dt).abs().t().contiguous()
    # fp32 sums of K / 32 products' sums and r of them, in runs of at most 16 and trees: some 40 roundings a term
    tol = 64 * 2.0 ** -24 * size
    ws = garbage(B.mmvq_lora_workspace(s, n))
    out = nan(n, M + 3)
    announce(f"lora {n} rows type {kind} rank {r}")
    B.mmvq_lora(s, x, K + 4, n, None, ids, n, base, M + 1, out, M + 3, ws, ws.numel())
    assert bool(((out[:, :M].double() - want).abs() <= tol).all()) and bool(out[:, M:].isnan().all())
    B.mmvq_lora(s, x, K + 4, n, None, ids, n, base, M + 1, base, M + 1, ws, ws.numel())
    assert torch.equal(base[:, :M], out[:, :M])
