"""Steps of a small server through all operators: requests come, grow and go
in a batch padded to a fixed number of rows, each with an adapter and settings
of its own. Every stage against its 64-bit form from what the stage before
gave, and the whole step as a replayed graph against the eager one."""
import numpy as np
import pytest

import decode_ref as D
import serve_ref as R
from gpu_helpers import dev, host
from quantized_decode_gemv_quantize_amd import binding as B
from quantized_decode_gemv_quantize_amd import synth

pytestmark = pytest.mark.gpu

K, V, H, HEADS, HD, PAGE, ROWS, SEQS, WIDE = 512, 1500, 2, 4, 64, 16, 24, 5, 12
QKV = (HEADS + 2 * H) * HD
EPS = 1e-5


class Server:
    """Buffers and descriptors of one copy of the server."""

    def __init__(self, weights, adapters, pool):
        import torch
        self.w, self.adapters = weights, adapters
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda:0")  # noqa: E731
        f32 = lambda *s: torch.zeros(s, device="cuda:0")  # noqa: E731
        u8 = lambda n: torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda:0")  # noqa: E731
        self.table, self.held, self.free, self.n_free = dev(pool.table), dev(pool.held), dev(pool.free), dev(np.array([pool.n_free], np.int32))
        self.pool = B.kv_pool(self.table, self.held, self.free, self.n_free, WIDE, pool.n_pages, PAGE)
        size = B.mmvq_kv_page_bytes(B.F16, PAGE, H, HD)
        self.cache = B.kv_cache(u8(pool.n_pages * size), u8(pool.n_pages * size), B.F16, pool.n_pages, PAGE, H, HD)
        self.keep, self.cached, self.new, self.start, self.len = i32(SEQS), i32(SEQS), i32(SEQS), i32(SEQS + 1), i32(SEQS)
        self.batch = B.kv_batch(self.start, self.len, self.table, SEQS, ROWS, ROWS, WIDE * PAGE, WIDE)
        self.seq, self.pos, self.missing, self.ids, self.adapter = i32(ROWS), i32(ROWS), i32(1), i32(ROWS), i32(SEQS)
        self.x, self.yq, self.qkv, self.q = f32(ROWS, K), u8(ROWS * K // 32 * 36), f32(ROWS, QKV), f32(ROWS, HEADS * HD)
        self.att, self.proj, self.logits, self.u = f32(ROWS, HEADS * HD), f32(ROWS, K), f32(ROWS, V), f32(ROWS)
        self.tokens, self.chosen, self.probs = i32(ROWS), f32(ROWS), f32(ROWS, V)
        self.T, self.k, self.p, self.m = f32(SEQS), i32(SEQS), f32(SEQS), f32(SEQS)
        self.settings = B.sampling(self.T, self.k, self.p, self.m)
        self.plan_ws, self.lora_ws = u8(B.mmvq_kv_plan_workspace(SEQS)), u8(B.mmvq_lora_workspace(adapters.set, ROWS))
        self.attn_ws, self.sample_ws = u8(B.mmvq_attn_workspace(self.cache, self.batch, HEADS) + 16), u8(B.mmvq_sample_workspace(ROWS, V))

    def step(self):
        w = self.w
        B.mmvq_kv_release(self.pool, SEQS, self.keep)
        B.mmvq_kv_plan(self.pool, self.cached, self.new, SEQS, ROWS, self.start, self.len, self.seq, self.pos, None, self.missing,
                       self.plan_ws, self.plan_ws.numel())
        B.mmvq_embed(w["table"], B.Q4_K, V, K, self.ids, ROWS, 1.5, self.x, K)
        B.mmvq_add_rms_norm(self.x, K, ROWS, K, None, 0, w["norm"], EPS, None, 0, None, 0, self.yq)
        B.mmvq(w["qkv"], B.Q8_0, QKV, K, self.yq, ROWS, self.qkv)
        B.mmvq_lora(self.adapters.set, self.x, K, ROWS, self.seq, self.adapter, SEQS, self.qkv, QKV, self.q, HEADS * HD, self.lora_ws,
                    self.lora_ws.numel())
        B.mmvq_kv_write(self.cache, self.batch, self.qkv[:, HEADS * HD:], QKV, self.qkv[:, (HEADS + H) * HD:], QKV)
        B.mmvq_attn(self.cache, self.batch, self.q, HEADS * HD, HEADS, HD ** -0.5, 0, None, self.att, HEADS * HD, self.attn_ws,
                    self.attn_ws.numel())
        B.mmvq_f32(w["o"], B.Q8_0, K, HEADS * HD, self.att, ROWS, HEADS * HD, self.proj)
        B.mmvq_add_rms_norm(self.proj, K, ROWS, K, self.x, K, None, EPS, None, 0, None, 0, self.yq)
        B.mmvq(w["table"], B.Q4_K, V, K, self.yq, ROWS, self.logits)     # the tied head
        B.mmvq_sample(self.logits, V, V, ROWS, self.settings, self.seq, SEQS, self.u, self.tokens, self.chosen, self.probs, V, self.sample_ws,
                      self.sample_ws.numel())

    OUT = ("table", "held", "free", "n_free", "start", "len", "seq", "pos", "x", "qkv", "q", "att", "logits", "tokens", "chosen", "probs")

    def snapshot(self):
        return {k: host(getattr(self, k)).copy() for k in self.OUT}


class Adapters:
    def __init__(self, rng):
        import torch
        self.A = torch.from_numpy(rng.standard_normal((3, 16, K)).astype(np.float32) / K ** 0.5).to(torch.bfloat16)
        self.B = torch.from_numpy(rng.standard_normal((3, HEADS * HD, 16)).astype(np.float32) * 0.1).to(torch.bfloat16)
        self.ranks, self.scales = np.array([16, 8, 5]), np.array([1.0, 2.0, 0.5], np.float32)
        self.set = B.lora_set(self.A.to("cuda:0"), self.B.to("cuda:0"), B.BF16, 3, K, HEADS * HD, 16, dev(self.ranks.astype(np.int32)),
                              dev(self.scales))


def test_server_steps():
    import torch
    rng = np.random.default_rng(33)
    weights = {"qkv": dev(synth.weights(B.Q8_0, QKV, K, rng)), "o": dev(synth.weights(B.Q8_0, K, HEADS * HD, rng)),
               "norm": dev((1 + 0.1 * rng.standard_normal(K)).astype(np.float32))}
    table = synth.weights(B.Q4_K, V, K, rng)
    weights["table"] = dev(table)
    rows = table.reshape(V, -1)
    adapters = Adapters(rng)
    pool = R.Pool(SEQS, WIDE, 34, PAGE, 34, rng)
    eager, captured = Server(weights, adapters, pool), Server(weights, adapters, pool)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        captured.step()                         # a step without new tokens: nothing of the pool changes
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            captured.step()
    torch.cuda.synchronize()

    history = [[] for _ in range(SEQS)]         # keys and values of each request's tokens, as the cache holds them
    last = np.zeros(SEQS, np.int64)
    for step in range(7):
        # requests end, new ones come in their places with a prompt, some wait, the others go on by one
        keep, new, ids = np.full(SEQS, -1), np.zeros(SEQS, int), []
        for s in range(SEQS):
            fresh = not history[s]
            if not fresh and rng.random() < 0.25:
                history[s], keep[s], fresh = [], 0, True
            if fresh:
                new[s] = rng.integers(1, 9) if rng.random() < 0.7 or step == 0 else 0
            else:
                new[s] = rng.random() < 0.9
        cached = np.array([len(h) for h in history])
        for s in range(SEQS):
            ids += list(rng.integers(0, V, new[s])) if cached[s] == 0 else [last[s]] * new[s]
        ids = np.array(ids + [-1] * (ROWS - len(ids)))[:ROWS]
        drawn = {"T": np.array([0.0, 0.8, 1.0, 1.2, 0.7]), "k": np.array([0, 30, 0, 0, 5]), "p": np.array([1.0, 0.9, 0.95, 1.0, 1.0]),
                 "m": np.array([0.0, 0.0, 0.0, 0.05, 0.0])}
        given = {"keep": keep, "cached": cached, "new": new, "ids": ids, "adapter": rng.integers(-1, 3, SEQS), "u": rng.random(ROWS), **drawn}
        for server in (eager, captured):
            for name, value in given.items():
                t = getattr(server, name)
                t.copy_(dev(np.asarray(value).astype(np.int32 if t.dtype == torch.int32 else np.float32)))
        eager.step()
        got = eager.snapshot()
        graph.replay()
        torch.cuda.synchronize()
        replayed = captured.snapshot()
        for key in got:
            assert np.array_equal(got[key], replayed[key]), (step, key)

        # pages and maps
        pool.release(keep)
        start, length, seq, pos, _, missing = pool.plan(cached, new, ROWS)
        assert missing == 0
        for key, want in (("start", start), ("len", length), ("seq", seq), ("pos", pos), ("table", pool.table), ("held", pool.held)):
            assert np.array_equal(got[key], want), (step, key)
        n = start[-1]
        # rows of the table
        want = np.stack([R.table_row(rows[i], B.Q4_K) * 1.5 if i >= 0 else np.zeros(K) for i in ids])
        assert (np.abs(got["x"] - want) <= np.abs(want) * R.U * (1 + 1e-6) + 2.0 ** -150).all()
        # adapters beside the queries' part of the projection
        owner = np.where(seq >= 0, given["adapter"][np.maximum(seq, 0)], -1)
        want, tol = R.lora(adapters.A.float().numpy(), adapters.B.float().numpy(), adapters.ranks, adapters.scales, got["x"],
                           got["qkv"][:, :HEADS * HD], owner, 1)
        assert (np.abs(got["q"] - want) <= tol).all()
        # attention over everything that the requests have said
        for s in range(SEQS):
            for r in range(start[s], start[s + 1]):
                kv = got["qkv"][r, HEADS * HD:].reshape(2, H, HD)
                history[s].append(D.stored(kv, "f16"))
            if new[s]:
                hk = np.stack(history[s])
                mine = slice(start[s], start[s + 1])
                ref, mag, smax = D.attention(got["q"][mine].reshape(-1, HEADS, HD), hk[:, 0], hk[:, 1], HD ** -0.5, cached[s])
                tol = D.attention_tolerance(ref, mag, smax, hk[:, 1], HD)
                assert (np.abs(got["att"][mine].reshape(-1, HEADS, HD) - ref) <= tol).all()
        # the next tokens
        for r in range(ROWS):
            if seq[r] < 0:
                assert got["tokens"][r] == -1 and got["chosen"][r] == 0 and not got["probs"][r].any()
                continue
            s = seq[r]
            w = R.distribution(got["logits"][r], drawn["T"][s], drawn["k"][s], drawn["p"][s], drawn["m"][s])
            assert got["tokens"][r] == R.drawn(w, np.float32(given["u"][r]))
            assert (np.abs(got["probs"][r] - w / w.sum()) <= w / w.sum() * R.U * (1 + 1e-4) + 2.0 ** -150).all()
        for s in range(SEQS):
            if new[s]:
                last[s] = got["tokens"][start[s + 1] - 1]
        assert n == new.sum()


def test_filtered_rows_verify_drafts():
    """The distributions that mmvq_sample leaves, as targets and as the draft's, in mmvq_verify_draft."""
    rng = np.random.default_rng(34)
    n, v, starts = 9, 3000, np.array([0, 4, 5, 9], np.int32)
    owner = dev(np.array([0, 0, 0, 0, 1, 2, 2, 2, 2], np.int32))
    z = [(rng.standard_normal((n, v)) * 3).astype(np.float32) for _ in "td"]
    z[1] = z[0] + 0.3 * z[1]
    T, p = np.array([0.7, 0.0, 1.1], np.float32), np.array([0.9, 1.0, 0.95], np.float32)
    import torch
    ws = torch.empty(B.mmvq_sample_workspace(n, v), dtype=torch.uint8, device="cuda:0")
    probs, tokens = [], torch.zeros(n, dtype=torch.int32, device="cuda:0")
    for rows, out in ((z[0], None), (z[1], tokens)):
        probs.append(dev(rows))                  # in place
        u = dev(rng.random(n, np.float32))
        B.mmvq_sample(probs[-1], v, v, n, B.sampling(dev(T), None, dev(p), None), owner, 3, u, out, None, probs[-1], v, ws, ws.numel())
    ua, us = rng.random(n, np.float32), rng.random(3, np.float32)
    count, out = torch.zeros(3, dtype=torch.int32, device="cuda:0"), torch.zeros((3, 4), dtype=torch.int32, device="cuda:0")
    vws = torch.empty(B.mmvq_verify_workspace(3, n, v), dtype=torch.uint8, device="cuda:0")
    B.mmvq_verify_draft(probs[0], v, v, B.TARGET_WEIGHTS, None, tokens, probs[1], v, dev(starts), 3, n, dev(ua), dev(us), count, out, 4, vws,
                        vws.numel())
    ec, eo = D.verify(host(probs[0]), B.TARGET_WEIGHTS, None, host(tokens), host(probs[1]), starts, ua, us, 4)
    assert np.array_equal(host(count), ec) and np.array_equal(host(out), eo) and ec.sum() > 0
