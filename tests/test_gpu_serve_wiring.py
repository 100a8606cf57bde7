"""Adapters where a model has them: beside the projections of the normed rows,
which mmvq_add_rms_norm hands on as q8_1 columns to the product and as fp32
ones to the adapter, and in place on what the product left; the last rows'
tokens drawn from the head's logits. Every stage against its 64-bit form from
what the stage before gave, eager and as a replayed graph."""
import numpy as np
import pytest

import oracle
import serve_ref as R
from gpu_helpers import REL, ABS, dev, host
from quantized_decode_gemv_quantize_amd import binding as B
from quantized_decode_gemv_quantize_amd import synth

pytestmark = pytest.mark.gpu

K, M, V, ROWS, SEQS, RANK, COUNT = 512, 768, 1000, 7, 4, 24, 3
EPS = 1e-5


class Layer:
    def __init__(self, weights, sets):
        import torch
        self.w, self.sets = weights, sets
        f32 = lambda *s: torch.zeros(s, device="cuda:0")  # noqa: E731
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda:0")  # noqa: E731
        u8 = lambda n: torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda:0")  # noqa: E731
        self.ids, self.seq, self.adapter = i32(ROWS), i32(ROWS), i32(SEQS)
        self.x, self.y, self.yq = f32(ROWS, K), f32(ROWS, K), u8(ROWS * K // 32 * 36)
        self.up, self.plain, self.down, self.h, self.logits, self.u = f32(ROWS, M), f32(ROWS, M), f32(ROWS, K), f32(ROWS, K), f32(ROWS, V), f32(ROWS)
        self.plain_down, self.z, self.zq = f32(ROWS, K), f32(ROWS, K), u8(ROWS * K // 32 * 36)
        self.tokens, self.chosen = i32(ROWS), f32(ROWS)
        self.ws = u8(max(B.mmvq_lora_workspace(s, ROWS) for s in sets))
        self.sample_ws = u8(B.mmvq_sample_workspace(ROWS, V))
        self.settings = B.sampling(dev(np.array([0.0, 0.8, 1.0, 1.2], np.float32)), dev(np.array([0, 30, 0, 0], np.int32)),
                                   dev(np.array([1.0, 0.9, 0.95, 1.0], np.float32)), None)

    def step(self):
        w = self.w
        B.mmvq_embed(w["table"], B.Q4_K, V, K, self.ids, ROWS, 1.5, self.x, K)
        B.mmvq_add_rms_norm(self.x, K, ROWS, K, None, 0, w["norm"], EPS, None, 0, self.y, K, self.yq)
        B.mmvq(w["up"], B.Q8_0, M, K, self.yq, ROWS, self.up)
        self.plain.copy_(self.up)
        B.mmvq_lora(self.sets[0], self.y, K, ROWS, self.seq, self.adapter, SEQS, self.up, M, self.up, M, self.ws, self.ws.numel())
        B.mmvq_f32(w["down"], B.Q8_0, K, M, self.up, ROWS, M, self.down)
        self.plain_down.copy_(self.down)
        B.mmvq_lora(self.sets[1], self.up, M, ROWS, self.seq, self.adapter, SEQS, self.down, K, self.down, K, self.ws, self.ws.numel())
        B.mmvq_add_rms_norm(self.down, K, ROWS, K, self.x, K, w["norm"], EPS, self.h, K, self.z, K, self.zq)
        B.mmvq(w["table"], B.Q4_K, V, K, self.zq, ROWS, self.logits)
        B.mmvq_sample(self.logits, V, V, ROWS, self.settings, self.seq, SEQS, self.u, self.tokens, self.chosen, None, V, self.sample_ws,
                      self.sample_ws.numel())

    OUT = ("x", "y", "yq", "plain", "up", "plain_down", "down", "h", "z", "zq", "logits", "tokens", "chosen")

    def snapshot(self):
        return {k: host(getattr(self, k)).copy() for k in self.OUT}


def norm64(x, weight):
    x = x.astype(np.float64)
    return x / np.sqrt((x * x).mean(1, keepdims=True) + np.float64(np.float32(EPS))) * weight.astype(np.float64)


def test_adapters_beside_the_normed_projections():
    import torch
    rng = np.random.default_rng(71)
    host_w = {"up": synth.weights(B.Q8_0, M, K, rng), "down": synth.weights(B.Q8_0, K, M, rng), "table": synth.weights(B.Q4_K, V, K, rng),
              "norm": (1 + 0.1 * rng.standard_normal(K)).astype(np.float32)}
    weights = {k: dev(v) for k, v in host_w.items()}
    ranks, scales = np.array([24, 7, 16]), np.array([1.0, 2.0, 0.5], np.float32)
    bf16 = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32) * 0.05).to(torch.bfloat16)  # noqa: E731
    mats = [(bf16(COUNT, RANK, K), bf16(COUNT, M, RANK)), (bf16(COUNT, RANK, M), bf16(COUNT, K, RANK))]
    sets = [B.lora_set(a.to("cuda:0"), b.to("cuda:0"), B.BF16, COUNT, a.shape[2], b.shape[1], RANK, dev(ranks.astype(np.int32)), dev(scales))
            for a, b in mats]
    eager, captured = Layer(weights, sets), Layer(weights, sets)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured.step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            captured.step()
    torch.cuda.synchronize()
    O = oracle.default()
    for step in range(4):
        ids = rng.integers(0, V, ROWS)
        seq = np.sort(rng.integers(0, SEQS, ROWS))
        if step:
            ids[-step:], seq[-step:] = -1, -1     # rows behind the last request
        given = {"ids": ids, "seq": seq, "adapter": rng.integers(-1, COUNT, SEQS), "u": rng.random(ROWS)}
        for layer in (eager, captured):
            for name, value in given.items():
                t = getattr(layer, name)
                t.copy_(dev(np.asarray(value).astype(np.int32 if t.dtype == torch.int32 else np.float32)))
        eager.step()
        got = eager.snapshot()
        graph.replay()
        torch.cuda.synchronize()
        replayed = captured.snapshot()
        for key in got:
            assert np.array_equal(got[key], replayed[key]), (step, key)
        owner = np.where(seq >= 0, given["adapter"][np.maximum(seq, 0)], -1)
        # the norm's fp32 output, rounded once, beside the q8_1 columns of the same values
        want = norm64(got["x"], host_w["norm"])
        assert (np.abs(got["y"] - want) <= np.abs(want) * R.U * (1 + 1e-6) + 2.0 ** -150).all()
        want = norm64(got["h"], host_w["norm"])
        assert (np.abs(got["z"] - want) <= np.abs(want) * R.U * (1 + 1e-6) + 2.0 ** -150).all()
        assert np.array_equal(got["h"], got["down"] + got["x"])
        # products of the q8_1 columns
        for name, src, kind, rows, cols, out in (("up", "yq", B.Q8_0, M, K, "plain"), ("table", "zq", B.Q4_K, V, K, "logits")):
            ref, mag, _ = O.mmvq(host_w[name], kind, rows, cols, got[src].reshape(ROWS, -1), ROWS)
            assert (np.abs(got[out].astype(np.float64) - ref) <= REL * mag + ABS).all(), (step, name)
        # adapters on what the products left, from the normed rows and from the rows between
        for (a, b), src, plain, out in ((mats[0], "y", "plain", "up"), (mats[1], "up", "plain_down", "down")):
            want, tol = R.lora(a.float().numpy(), b.float().numpy(), ranks, scales, got[src], got[plain], owner, 1)
            assert (np.abs(got[out] - want) <= tol).all(), (step, out)
            assert step == 0 or np.array_equal(got[out][owner < 0], got[plain][owner < 0])
        for r in range(ROWS):
            s = seq[r]
            w = np.zeros(V)
            if s >= 0:
                w = R.distribution(got["logits"][r], [0.0, 0.8, 1.0, 1.2][s], [0, 30, 0, 0][s], [1.0, 0.9, 0.95, 1.0][s])
            assert got["tokens"][r] == R.drawn(w, np.float32(given["u"][r]))
