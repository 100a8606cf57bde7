"""Cases of the operators of a step over many requests: the pages of finished
requests given back and the next step's tables and maps built from the
requests' lengths, the tokens' rows of an embedding table, the requests'
low-rank adapters beside a shared projection, and the next tokens drawn from
the logits, with the probability that each was drawn with.

Block layouts of the table types (bytes; d, m, dmin are fp16):

  q4_0  18 / 32    d @0, nibbles @2; value d (q - 8)
  q4_1  20 / 32    d @0, m @2, nibbles @4; value d q + m
  q5_0  22 / 32    d @0, fifth bits @2, nibbles @6; value d (q - 16)
  q5_1  24 / 32    d @0, m @2, fifth bits @4, nibbles @8; value d q + m
  q8_0  34 / 32    d @0, int8 codes @2; value d q
  q4_k  144 / 256  d @0, dmin @2, 6-bit scales and mins @4, nibbles @16;
                   value d sc q - dmin m
  q5_k  176 / 256  the same with fifth bits @16 and nibbles @48
  q6_k  210 / 256  low bits @0, high bits @128, int8 scales @192, d @208;
                   value d sc (q - 32)

Nibble j of the 32-value blocks is value j (low) and j + 16 (high); chunk c of
64 values of q4_k and q5_k has bytes 32 c .. 32 c + 31, the low nibbles its
first 32 values.
"""
import math
import random
import struct

import numpy as np
import torch

own = False

DEV = "cuda"
TYPE_ID = {"f32": 0, "f16": 1, "q4_0": 2, "q4_1": 3, "q5_0": 6, "q5_1": 7, "q8_0": 8, "q4_k": 12, "q5_k": 13, "q6_k": 14,
           "bf16": 30}
FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = {"q4_0": (32, 18), "q4_1": (32, 20), "q5_0": (32, 22), "q5_1": (32, 24), "q8_0": (32, 34), "q4_k": (256, 144),
         "q5_k": (256, 176), "q6_k": (256, 210), "f32": (1, 4), "f16": (1, 2), "bf16": (1, 2)}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one user's token, a table that is also the language-model head
        {"name": "embed_1_q6k", "op": "embed", "type": "q6_k", "vocab": 128256, "K": 4096, "n": 1, "scale": 1.0},
        # a short prompt beside other users' tokens, a table in 16 bits with an odd row length
        {"name": "embed_777_bf16", "op": "embed", "type": "bf16", "vocab": 50257, "K": 2565, "n": 777, "scale": 1.0},
        # a prompt's chunk of 4096 tokens, rows scaled by the root of their length
        {"name": "embed_4096_q4k", "op": "embed", "type": "q4_k", "vocab": 128256, "K": 4096, "n": 4096, "scale": 64.0},
        # one user's token through its adapter beside the output projection
        {"name": "lora_1", "op": "lora", "type": "bf16", "K": 4096, "M": 4096, "max_rank": 16, "ranks": "equal", "adapters": 4,
         "requests": 1, "n": 1, "pad": 0},
        # 64 users' tokens, each with one of 100 adapters of unlike ranks or none, beside the up projection
        {"name": "lora_64_mixed", "op": "lora", "type": "f16", "K": 4096, "M": 14336, "max_rank": 64, "ranks": "mixed", "adapters": 100,
         "requests": 64, "n": 64, "pad": 0},
        # chunks of eight users' prompts beside the down projection, rows padded to a graph's batch
        {"name": "lora_prompts", "op": "lora", "type": "bf16", "K": 14336, "M": 4096, "max_rank": 32, "ranks": "equal", "adapters": 6,
         "requests": 8, "n": 4000, "pad": 96},
        # a step of 64 users: single and drafted tokens, some requests replaced by short new ones
        {"name": "pages_64", "op": "pages", "page": 16, "requests": 64, "new": 4, "chunk": 100, "fresh": 3, "len": 4000, "pad": 17},
        # a step of 512 requests, 40 of them new with prompts of up to 2000 tokens
        {"name": "pages_512_prompts", "op": "pages", "page": 32, "requests": 512, "new": 1, "chunk": 2000, "fresh": 40, "len": 6000, "pad": 0},
        # one user's next token: temperature and all three filters
        {"name": "sample_1", "op": "sample", "vocab": 128256, "rows": 1, "requests": 1, "filters": "all", "probs": False, "masked": 0.0},
        # 64 users, each with settings of its own: greedy, plain, filtered
        {"name": "sample_64_mixed", "op": "sample", "vocab": 128256, "rows": 64, "requests": 64, "filters": "mixed", "probs": False, "masked": 0.0},
        # the filtered distributions of 32 users' 128 drafted rows, for their verification
        {"name": "sample_128_probs", "op": "sample", "vocab": 128256, "rows": 128, "requests": 32, "filters": "top_p", "probs": True, "masked": 0.0},
        # 256 users, most of whose vocabulary a grammar or a language rules out; a vocabulary that no tile divides
        {"name": "sample_256_masked", "op": "sample", "vocab": 151669, "rows": 256, "requests": 256, "filters": "mixed", "probs": False, "masked": 0.7},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["embed", "lora", "lora", "pages", "sample", "sample"])
    if op == "embed":
        kind = rng.choice(sorted(TYPE_ID))
        qk = BLOCK[kind][0]
        K = qk * _log_int(rng, max(1, -(-128 // qk)), 14336 // qk)
        return {"op": "embed", "type": kind, "vocab": _log_int(rng, 1000, min(128256, 2 ** 29 // K)), "K": K,
                "n": _log_int(rng, 1, min(8192, 2 ** 24 // K)), "scale": rng.choice([1.0, round(math.sqrt(K), 2)])}
    if op == "lora":
        n = _log_int(rng, 1, 4096)
        K, M, rank = 32 * _log_int(rng, 8, 448), _log_int(rng, 200, 14336), 8 * _log_int(rng, 1, 16)
        while n * rank * (K + M) > 2 ** 31:
            n = max(1, n // 2)
        most = max(1, min(128, 2 ** 29 // (rank * (K + M))))
        return {"op": "lora", "type": rng.choice(sorted(FLOATS)), "K": K, "M": M, "max_rank": rank, "ranks": rng.choice(["equal", "mixed"]),
                "adapters": _log_int(rng, 1, most), "requests": _log_int(rng, 1, min(n, 128)), "n": n, "pad": rng.choice([0, rng.randint(0, 40)])}
    if op == "pages":
        requests = _log_int(rng, 1, 512)
        return {"op": "pages", "page": rng.choice([16, 32, 64, 128]), "requests": requests, "new": rng.randint(1, 8),
                "chunk": _log_int(rng, 1, 2000), "fresh": rng.randint(0, min(requests, 40)), "len": _log_int(rng, 10, 6000),
                "pad": rng.choice([0, rng.randint(0, 64)])}
    requests = _log_int(rng, 1, 64)
    return {"op": "sample", "vocab": _log_int(rng, 1000, 151669), "rows": min(256, requests * rng.choice([1, 1, 1, 2, 5])), "requests": requests,
            "filters": rng.choice(["all", "mixed", "top_p", "top_k", "min_p", "none"]), "probs": rng.random() < 0.3,
            "masked": rng.choice([0.0, 0.0, 0.5, 0.99])}


def _row_bytes(case):
    qk, size = BLOCK[case["type"]]
    return case["K"] // qk * size


def _rank_list(case):
    r, most = random.Random(case["adapters"] * 31 + case["max_rank"]), case["max_rank"]
    if case["ranks"] == "equal":
        return [most] * case["adapters"]
    return [most] + [r.choice([most, max(1, most // 2), max(1, most // 4), r.randint(1, most)]) for _ in range(case["adapters"] - 1)]


def _assigned(case):
    """Rows of each request, and its adapter (-1: none; the first request has one)."""
    r = random.Random(case["n"] * 7 + case["requests"])
    cuts = sorted(r.sample(range(1, case["n"]), case["requests"] - 1))
    rows = [b - a for a, b in zip([0] + cuts, cuts + [case["n"]])]
    return rows, [0] + [r.randint(0, case["adapters"] - 1) if r.random() < 0.85 else -1 for _ in range(case["requests"] - 1)]


def _lens(case):
    """Per request: tokens in the cache before the step, new ones, and the pages that it keeps (-1: all of them)."""
    r = random.Random(case["requests"] * 1009 + case["len"] * 7 + case["page"])
    fresh = set(r.sample(range(case["requests"]), case["fresh"]))
    got = []
    for s in range(case["requests"]):
        if s in fresh:
            got.append((0, r.randint(max(1, case["chunk"] // 2), case["chunk"]), 0))
            continue
        cached, new = r.randint(max(1, case["len"] // 3), case["len"]), r.randint(0 if s else 1, case["new"])
        held = -(-cached // case["page"])
        got.append((cached, new, held if new and held * case["page"] < cached + new else -1))
    return got


def work(case):
    if case["op"] == "embed":
        return {"bytes": case["n"] * (_row_bytes(case) + 4 * case["K"] + 4), "flops": case["n"] * case["K"] * 2}
    if case["op"] == "lora":
        rows, ids = _assigned(case)
        ranks, size = _rank_list(case), BLOCK[case["type"]][1]
        weights = sum(ranks[a] for a in set(ids) - {-1}) * (case["K"] + case["M"]) * size
        flops = sum(2 * n * ranks[a] * (case["K"] + case["M"]) for n, a in zip(rows, ids) if a >= 0)
        moved = sum(n for n, a in zip(rows, ids) if a >= 0) * case["K"] * 4 + (case["n"] + case["pad"]) * case["M"] * 8
        return {"bytes": weights + moved, "flops": flops}
    if case["op"] == "pages":
        lens = _lens(case)
        rows = sum(n for _, n, _ in lens) + case["pad"]
        pages = sum(-(-(c + n) // case["page"]) - k for c, n, k in lens if k >= 0)
        return {"bytes": rows * 16 + len(lens) * 28 + pages * 16, "flops": rows * 8}
    moved = case["rows"] * case["vocab"] * (8 if case["probs"] else 4)
    return {"bytes": moved, "flops": case["rows"] * case["vocab"] * 4}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(DEV).manual_seed(seed * 2 + 1)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV)


def _table(g, kind, vocab, K):
    """Rows of values of some 0.02: random codes, scales by the type."""
    if kind in FLOATS:
        return (_normal(g, vocab, K) * 0.02).to(FLOATS[kind])
    qk, size = BLOCK[kind]
    t = torch.randint(0, 256, (vocab, K // qk, size), generator=g, device=DEV, dtype=torch.uint8)
    steps = {"q4_0": 8, "q4_1": 8, "q5_0": 16, "q5_1": 16, "q8_0": 64, "q4_k": 256, "q5_k": 512, "q6_k": 1024}[kind]
    for at in {"q6_k": [208], "q4_1": [0, 2], "q5_1": [0, 2], "q4_k": [0, 2], "q5_k": [0, 2]}.get(kind, [0]):
        offset = at == 2 and kind in ("q4_1", "q5_1")
        d = (_uniform(g, vocab, K // qk, 1) + 0.5) * (-0.02 if offset else 0.02 / steps)
        t[..., at:at + 2] = d.half().view(torch.uint8)
    return t.view(vocab, -1)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _settings(case, seed):
    """Temperature, top-k, top-p, min-p of each request; what is off has the value that says so."""
    r, n, got = random.Random(seed * 11 + 5), case["requests"], []
    for _ in range(n):
        T, k, p, m = r.uniform(0.5, 1.3), r.choice([20, 40, 64, 200]), r.uniform(0.8, 0.98), r.uniform(0.01, 0.1)
        what = case["filters"]
        if what == "mixed":
            what = r.choice(["greedy", "none", "top_k", "top_p", "min_p", "all"])
        got.append((0.0 if what == "greedy" else T, k if what in ("all", "top_k") else 0, p if what in ("all", "top_p") else 1.0,
                    m if what in ("all", "min_p") else 0.0))
    T, k, p, m = zip(*got)
    return [torch.tensor(x, dtype=torch.float32, device=DEV) for x in (T, p, m)] + [_ints(k)]


def prepare(case, seed):
    g, s = _gen(seed), {"case": case}
    if case["op"] == "embed":
        s["table"] = _table(g, case["type"], case["vocab"], case["K"])
        s["ids"] = torch.randint(0, case["vocab"], (case["n"],), generator=g, device=DEV, dtype=torch.int32)
        s["out"] = torch.empty(case["n"], case["K"], device=DEV)
        s["scale"] = struct.unpack("f", struct.pack("f", case["scale"]))[0]
    elif case["op"] == "lora":
        rows, ids = _assigned(case)
        ranks, n, R = _rank_list(case), case["n"] + case["pad"], case["max_rank"]
        s["A"] = (_normal(g, case["adapters"], R, case["K"]) / math.sqrt(case["K"])).to(FLOATS[case["type"]])
        s["B"] = (_normal(g, case["adapters"], case["M"], R) * 0.1).to(FLOATS[case["type"]])
        s["rank"], s["scale"] = _ints(ranks), torch.tensor([32.0 / r for r in ranks], device=DEV)
        s["x"], s["y"] = _normal(g, n, case["K"]), _normal(g, n, case["M"])
        owner = np.concatenate([np.repeat(np.arange(len(rows)), rows), np.full(case["pad"], -1)])
        s["row_seq"], s["adapter"] = _ints(owner.tolist()), _ints(ids)
        s["out"] = torch.empty(n, case["M"], device=DEV)
        # the rows of each adapter and its rank, as the program that made the batch knows them
        of_row = np.where(owner >= 0, np.array(ids)[owner], -1)
        s["groups"] = [(a, ranks[a], torch.from_numpy(np.flatnonzero(of_row == a)).to(DEV)) for a in sorted(set(ids) - {-1})]
    elif case["op"] == "pages":
        lens, page = _lens(case), case["page"]
        need = [-(-(c + n) // page) for c, n, _ in lens]
        s["wide"], s["n_pages"] = max(need) + 2, sum(need) + 50
        order = np.random.RandomState(seed % (1 << 31)).permutation(s["n_pages"]).astype(np.int32)
        table, at = np.full((len(lens), s["wide"]), -1, dtype=np.int32), 0
        for i, k in enumerate(need):
            table[i, :k] = order[at:at + k]
            at += k
        free = np.full(s["n_pages"], -1, dtype=np.int32)
        free[:50] = order[at:]
        s["table"], s["free"], s["n_free"] = torch.from_numpy(table).to(DEV), torch.from_numpy(free).to(DEV), _ints([50])
        s["held"] = _ints(need)
        s["cached"], s["new"], s["keep"] = (_ints(list(x)) for x in zip(*lens))
        s["rows"] = sum(n for _, n, _ in lens) + case["pad"]
        empty = lambda n, t: torch.empty(n, dtype=t, device=DEV)
        s["start"], s["len"], s["missing"] = (empty(n, torch.int32) for n in (len(lens) + 1, len(lens), 1))
        s["row_seq"], s["row_pos"], s["row_slot"] = (empty(s["rows"], t) for t in (torch.int32, torch.int32, torch.int64))
    else:
        n, V = case["rows"], case["vocab"]
        # a language-model head's logits: a few likely tokens above a broad floor
        x = _normal(g, n, V) * 2.0
        x.scatter_add_(1, torch.randint(0, V, (n, 300), generator=g, device=DEV), _uniform(g, n, 300) * 14.0)
        if case["masked"]:
            x.masked_fill_(_uniform(g, n, V) < case["masked"], -math.inf)
        s["logits"], s["u"] = x, _uniform(g, n)
        s["T"], s["p"], s["m"], s["k"] = _settings(case, seed)
        owner = [i * case["requests"] // n for i in range(n)]
        s["row_seq"] = None if n == case["requests"] else _ints(owner)
        s["owner"] = torch.tensor(owner, device=DEV)
        s["tokens"], s["chosen"] = torch.empty(n, dtype=torch.int32, device=DEV), torch.empty(n, device=DEV)
        s["probs"] = torch.empty(n, V, device=DEV) if case["probs"] else None
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        return {"embed": _own_embed, "lora": _own_lora, "pages": _own_pages, "sample": _own_sample}[case["op"]](s, case)
    return {"embed": _embed, "lora": _lora, "pages": _pages, "sample": _sample}[case["op"]](s, case)


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV)


def _own_embed(s, c):
    from quantized_decode_gemv_quantize_amd import binding as B
    B.mmvq_embed(s["table"], TYPE_ID[c["type"]], c["vocab"], c["K"], s["ids"], c["n"], s["scale"], s["out"], c["K"])
    return s["out"]


def _own_lora(s, c):
    from quantized_decode_gemv_quantize_amd import binding as B
    n = c["n"] + c["pad"]
    if "set" not in s:
        s["set"] = B.lora_set(s["A"], s["B"], TYPE_ID[c["type"]], c["adapters"], c["K"], c["M"], c["max_rank"], s["rank"], s["scale"])
        s["ws"] = _bytes(B.mmvq_lora_workspace(s["set"], n))
    B.mmvq_lora(s["set"], s["x"], c["K"], n, s["row_seq"], s["adapter"], c["requests"], s["y"], c["M"], s["out"], c["M"], s["ws"],
                s["ws"].numel())
    return s["out"]


def _own_pages(s, c):
    from quantized_decode_gemv_quantize_amd import binding as B
    n = c["requests"]
    if "pool" not in s:
        s["pool"] = B.kv_pool(s["table"], s["held"], s["free"], s["n_free"], s["wide"], s["n_pages"], c["page"])
        s["ws"] = _bytes(B.mmvq_kv_plan_workspace(n))
    B.mmvq_kv_release(s["pool"], n, s["keep"], None)
    B.mmvq_kv_plan(s["pool"], s["cached"], s["new"], n, s["rows"], s["start"], s["len"], s["row_seq"], s["row_pos"], s["row_slot"],
                   s["missing"], s["ws"], s["ws"].numel())
    return {k: s[k] for k in PAGES_OUT}


PAGES_OUT = ("table", "held", "free", "n_free", "start", "len", "row_seq", "row_pos", "row_slot", "missing")


def _own_sample(s, c):
    from quantized_decode_gemv_quantize_amd import binding as B
    n, V = c["rows"], c["vocab"]
    if "ws" not in s:
        s["set"] = B.sampling(s["T"], s["k"], s["p"], s["m"])
        s["ws"] = _bytes(B.mmvq_sample_workspace(n, V))
    B.mmvq_sample(s["logits"], V, V, n, s["set"], s["row_seq"], c["requests"], s["u"], s["tokens"], s["chosen"], s["probs"], V, s["ws"],
                  s["ws"].numel())
    return {"tokens": s["tokens"], "chosen": s["chosen"], "probs": s["probs"]}


def _half(blocks, at):
    return blocks[..., at:at + 2].contiguous().view(torch.float16).float()


def _nibbles(b):
    return torch.cat([b & 15, b >> 4], -1).float()


def _bits(b):
    """The bits of bytes [..., n], lowest first: [..., 8 n]."""
    return ((b[..., None] >> torch.arange(8, dtype=torch.uint8, device=DEV)) & 1).flatten(-2).float()


def _k_scales(b):
    """Scales and mins [..., 8, 1] of the 12 packed bytes."""
    lo, mid, hi = b[..., 0:4], b[..., 4:8], b[..., 8:12]
    sc = torch.cat([lo & 63, (hi & 15) | (lo >> 6 << 4)], -1)
    m = torch.cat([mid & 63, (hi >> 4) | (mid >> 6 << 4)], -1)
    return sc.float()[..., None], m.float()[..., None]


def _dequantized(rows, kind, K):
    """Rows of blocks -> values in 32 bits."""
    b = rows.view(rows.shape[0], -1, BLOCK[kind][1])
    if kind == "q6_k":
        ql = b[..., :128].unflatten(-1, (2, 2, 32))
        qh = b[..., 128:192].unflatten(-1, (2, 1, 32))
        low = torch.cat([ql & 15, ql >> 4], -2)
        high = (qh >> torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=DEV)[:, None]) & 3
        q = (low | (high << 4)).float().flatten(-3).unflatten(-1, (16, 16)) - 32.0
        sc = b[..., 192:208].contiguous().view(torch.int8).float()[..., None]
        return (_half(b, 208)[..., None] * sc * q).reshape(-1, K)
    if kind in ("q4_k", "q5_k"):
        sc, m = _k_scales(b[..., 4:16])
        at = 16 if kind == "q4_k" else 48
        q = _nibbles(b[..., at:at + 128].unflatten(-1, (4, 32))).unflatten(-1, (2, 32)).flatten(-3, -2)
        if kind == "q5_k":
            q = q + 16.0 * _bits(b[..., 16:48]).unflatten(-1, (32, 8)).transpose(-1, -2)
        return (_half(b, 0)[..., None] * sc * q - _half(b, 2)[..., None] * m).reshape(-1, K)
    d = _half(b, 0)
    if kind == "q8_0":
        return (d * b[..., 2:].contiguous().view(torch.int8).float()).reshape(-1, K)
    q = _nibbles(b[..., -16:])
    if kind in ("q5_0", "q5_1"):
        q = q + 16.0 * _bits(b[..., -20:-16])
    v = d * q + _half(b, 2) if kind in ("q4_1", "q5_1") else d * (q - (8.0 if kind == "q4_0" else 16.0))
    return v.reshape(-1, K)


def _embed(s, c):
    rows = s["table"][s["ids"].long()]
    v = rows.float() if c["type"] in FLOATS else _dequantized(rows, c["type"], c["K"])
    return v * s["scale"]


def _lora(s, c):
    n, R = c["n"] + c["pad"], c["max_rank"]
    if n <= 64 and n * R * (c["K"] + c["M"]) <= 2 ** 27:
        # each row's own copy of its adapter
        a = torch.where(s["row_seq"] >= 0, s["adapter"][s["row_seq"].clamp(min=0)], -1).long()
        at = a.clamp(min=0)
        v = torch.bmm(s["A"][at].float(), s["x"][:, :, None])
        v = torch.where(torch.arange(R, device=DEV)[:, None] < s["rank"][at][:, None, None], v, 0.0)
        y = torch.bmm(s["B"][at].float(), v)[:, :, 0] * s["scale"][at][:, None]
        return s["y"] + torch.where((a >= 0)[:, None], y, 0.0)
    out = s["y"].clone()
    for a, rank, rows in s["groups"]:
        v = s["x"][rows] @ s["A"][a, :rank].float().t()
        out[rows] += s["scale"][a] * (v @ s["B"][a, :, :rank].float().t())
    return out


def _pages(s, c):
    page, wide, held, free = c["page"], s["wide"], s["held"], s["free"]
    p = torch.arange(wide, device=DEV)
    # pages behind those kept go to the end of the free ones, in order
    left = torch.where(s["keep"] >= 0, torch.minimum(s["keep"], held), held)
    back = (p >= left[:, None]) & (p < held[:, None])
    at = torch.where(back.flatten(), s["n_free"] + back.flatten().cumsum(0) - 1, s["n_pages"])
    more = torch.cat([free, free[:1]])
    more[at] = s["table"].flatten()
    free.copy_(more[:-1])
    s["table"].masked_fill_(back, -1)
    s["n_free"] += back.sum()
    held.copy_(left)
    # lengths, and the pages that they need
    s["start"][:1] = 0
    s["start"][1:] = s["new"].cumsum(0)
    torch.add(s["cached"], s["new"], out=s["len"])
    need = torch.where(s["new"] > 0, torch.maximum(held, (s["len"] + page - 1) // page), held)
    want = (p >= held[:, None]) & (p < need[:, None])
    total = want.sum()
    given = torch.minimum(total, s["n_free"])
    nth = want.flatten().cumsum(0) - 1
    got = want.flatten() & (nth < given)
    took = free[torch.where(got, s["n_free"] - given + nth, 0)]
    s["table"].copy_(torch.where(got, took, s["table"].flatten()).view_as(s["table"]))
    held += got.view_as(want).sum(1).to(torch.int32)
    s["n_free"] -= given
    s["missing"][:] = total - given
    # each row's request, position and slot
    row = torch.arange(s["rows"], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["start"], row, right=True) - 1
    live = seq < c["requests"]
    seq = torch.where(live, seq, 0)
    pos = s["cached"][seq] + row - s["start"][seq]
    at = s["table"][seq, torch.where(live, pos // page, 0)].long()
    s["row_seq"].copy_(torch.where(live, seq, -1))
    s["row_pos"].copy_(torch.where(live, pos, -1))
    s["row_slot"].copy_(torch.where(live & (at >= 0), at * page + pos % page, -1))
    return {k: s[k] for k in PAGES_OUT}


def _sample(s, c):
    # 64 bits: a token goes by which side of a border of the running sum the given number lies on
    V, owner = c["vocab"], s["owner"]
    T, p, m, k = (s[name][owner][:, None] for name in "Tpmk")
    x = s["logits"].double()
    top, best = x.max(1, keepdim=True)
    e = torch.exp((x - top) / torch.where(T > 0, T, 1.0).double())
    e = torch.where(T > 0, e, torch.zeros_like(e).scatter_(1, best, 1.0))
    down, order = torch.sort(e, dim=1, descending=True, stable=True)
    # equal weights of unequal logits: the order is the logits' own
    order = torch.where(T > 0, torch.sort(x, dim=1, descending=True, stable=True)[1], order)
    down = e.gather(1, order)
    rank = torch.arange(V, device=DEV)
    down = torch.where((rank < k) | (k <= 0), down, 0.0)
    before = down.cumsum(1) - down
    keep = (before < p.double() * down.sum(1, keepdim=True)) | (p >= 1)
    keep &= down >= torch.where(m > 0, m.clamp(max=1.0), 0.0).double()
    keep[:, 0] = True
    e = torch.zeros_like(e).scatter_(1, order, torch.where(keep, down, 0.0))
    total = e.sum(1, keepdim=True)
    up = e.cumsum(1)
    hit = up > s["u"].double()[:, None] * total
    last = V - 1 - (e > 0).flip(1).to(torch.uint8).argmax(1)
    token = torch.where(hit.any(1), hit.to(torch.uint8).argmax(1), last)
    chosen = e.gather(1, token[:, None]) / total
    return {"tokens": token.to(torch.int32), "chosen": chosen[:, 0].float(), "probs": (e / total).float() if c["probs"] else None}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "lora": _exact_lora, "pages": _exact_pages, "sample": _exact_sample}[case["op"]](s, case)


def _exact_values(rows, kind, K):
    """Element by element: the block, byte and bits that hold each of a row's values."""
    qk, size = BLOCK[kind]
    i = np.arange(K)
    b, j = i // qk * size, i % qk
    byte = lambda at: rows[:, b + at].astype(np.int64)
    half = lambda at: (byte(at) | byte(at + 1) << 8).astype(np.uint16).view(np.float16).astype(np.float64)
    if kind == "q8_0":
        return half(0) * ((byte(2 + j) + 128) % 256 - 128)
    if kind == "q6_k":
        h, g, l = j // 128, j // 32 % 4, j % 32
        low = byte(64 * h + 32 * (g % 2) + l) >> (4 * (g // 2)) & 15
        high = byte(128 + 32 * h + l) >> (2 * g) & 3
        return half(208) * ((byte(192 + j // 16) + 128) % 256 - 128) * (low + 16 * high - 32)
    if kind in ("q4_k", "q5_k"):
        t, l, at = j // 32, j % 32, 16 if kind == "q4_k" else 48
        q = byte(at + 32 * (t // 2) + l) >> (4 * (t % 2)) & 15
        if kind == "q5_k":
            q = q + 16 * (byte(16 + l) >> t & 1)
        early = t < 4
        sc = np.where(early, byte(4 + t % 4) & 63, (byte(12 + t % 4) & 15) + 16 * (byte(4 + t % 4) >> 6))
        m = np.where(early, byte(8 + t % 4) & 63, (byte(12 + t % 4) >> 4) + 16 * (byte(8 + t % 4) >> 6))
        return half(0) * sc * q - half(2) * m
    q = byte(size - 16 + j % 16) >> (4 * (j // 16)) & 15
    if kind in ("q5_0", "q5_1"):
        q = q + 16 * (byte(size - 20 + j // 8) >> (j % 8) & 1)
    if kind in ("q4_1", "q5_1"):
        return half(0) * q + half(2)
    return half(0) * (q - (8 if kind == "q4_0" else 16))


def _exact_embed(s, c):
    rows = s["table"][s["ids"].long()]
    if c["type"] in FLOATS:
        return rows.double().cpu().numpy() * s["scale"]
    rows = rows.cpu().numpy()
    return np.concatenate([_exact_values(rows[i:i + 512], c["type"], c["K"]) for i in range(0, len(rows), 512)]) * s["scale"]


def _exact_lora(s, c):
    out = s["y"].double()
    owner, ids = s["row_seq"].cpu().numpy(), s["adapter"].cpu().numpy()
    first = 0
    while first < len(owner):                  # one request after the other
        last = first
        while last < len(owner) and owner[last] == owner[first]:
            last += 1
        a = ids[owner[first]] if owner[first] >= 0 else -1
        if a >= 0:
            r = int(s["rank"][a])
            part = torch.matmul(s["x"][first:last].double(), s["A"][a].double()[:r].t().contiguous())
            out[first:last] += float(s["scale"][a]) * torch.matmul(part, s["B"][a].double()[:, :r].t().contiguous())
        first = last
    return out


def _exact_pages(s, c):
    """One request after the other, one page after the other."""
    page, table, free = c["page"], s["table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    held, n_free = s["held"].cpu().numpy().copy(), int(s["n_free"][0])
    cached, new, keep = (s[k].cpu().numpy() for k in ("cached", "new", "keep"))
    for i in range(len(held)):
        if 0 <= keep[i] < held[i]:
            for p in range(keep[i], held[i]):
                free[n_free] = table[i, p]
                n_free += 1
                table[i, p] = -1
            held[i] = keep[i]
    wanted = [(i, p) for i in range(len(held)) if new[i] > 0 for p in range(held[i], -(-(cached[i] + new[i]) // page))]
    given = wanted[:n_free]
    for at, (i, p) in enumerate(given):
        table[i, p] = free[n_free - len(given) + at]
        held[i] += 1
    start = np.zeros(len(held) + 1, dtype=np.int32)
    seq, pos, slot = np.full(s["rows"], -1, np.int32), np.full(s["rows"], -1, np.int32), np.full(s["rows"], -1, np.int64)
    for i in range(len(held)):
        start[i + 1] = start[i] + new[i]
        for t in range(new[i]):
            r, at = start[i] + t, cached[i] + t
            seq[r], pos[r] = i, at
            if table[i, at // page] >= 0:
                slot[r] = int(table[i, at // page]) * page + at % page
    one = lambda v: np.array([v], dtype=np.int32)
    return {"table": table, "held": held, "free": free, "n_free": one(n_free - len(given)), "start": start,
            "len": (cached + new).astype(np.int32), "row_seq": seq, "row_pos": pos, "row_slot": slot, "missing": one(len(wanted) - len(given))}


def _exact_sample(s, c):
    """One row after the other, one filter after the other."""
    n, V = c["rows"], c["vocab"]
    tokens, chosen = np.empty(n, dtype=np.int32), np.empty(n)
    probs = np.zeros((n, V)) if c["probs"] else None
    T, top_p, min_p, top_k = (s[name].cpu().numpy().astype(np.float64)[s["owner"].cpu().numpy()] for name in "Tpmk")
    u = s["u"].cpu().numpy().astype(np.float64)
    for r in range(n):
        z = s["logits"][r].cpu().numpy().astype(np.float64)
        if T[r] > 0:
            w = np.exp((z - z.max()) / T[r])
        else:
            w = (np.arange(V) == z.argmax()).astype(np.float64)
        alive = np.flatnonzero(w > 0)
        alive = alive[np.lexsort((alive, -z[alive]))]       # falling logits, rising indices
        if top_k[r] > 0:
            alive = alive[:int(top_k[r])]
        if top_p[r] < 1:
            reached = np.cumsum(w[alive]) >= top_p[r] * w[alive].sum()
            alive = alive[:1 + int(reached.argmax())] if reached.any() else alive
        if min_p[r] > 0:
            alive = alive[w[alive] >= min(min_p[r], 1.0)]
        alive = np.sort(alive)
        up = np.cumsum(w[alive])
        hit = np.flatnonzero(up > u[r] * up[-1])
        tokens[r] = alive[hit[0] if len(hit) else -1]
        chosen[r] = w[tokens[r]] / w[alive].sum()
        if c["probs"]:
            probs[r, alive] = w[alive] / w[alive].sum()
    return {"tokens": tokens, "chosen": chosen, "probs": probs}
