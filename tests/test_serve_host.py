"""Operators of a step over many requests, without a GPU: declared and
exported, the host-only queries, and every refusal (arguments are checked
before any device is touched)."""
import ctypes
import gc
import os
import shutil
import subprocess
import weakref

import pytest

from quantized_decode_gemv_quantize_amd import binding as B

P, ODD = 1 << 20, (1 << 20) + 2     # never dereferenced


@pytest.fixture(scope="module")
def L():
    return B.lib()


def test_declared_symbols_are_exported_and_bound(L):
    names = B.declared_symbols(B.SERVE_HEADER)
    assert set(names) == {"mmvq_embed", "mmvq_kv_release", "mmvq_kv_plan_workspace", "mmvq_kv_plan", "mmvq_lora_workspace",
                          "mmvq_lora", "mmvq_sample_workspace", "mmvq_sample"}
    for n in names:
        assert hasattr(L, n) and n in B._SIGS and hasattr(B, n), n


EMBED = dict(table=P, kind=B.Q4_K, vocab=10, K=512, ids=P, n=3, scale=1.0, out=P, ldo=512)


@pytest.mark.parametrize("kw,code", [
    ({"table": None}, B.ERR_NULL), ({"ids": None}, B.ERR_NULL), ({"out": None}, B.ERR_NULL),
    ({"kind": B.Q8_1}, B.ERR_TYPE), ({"kind": 4}, B.ERR_TYPE), ({"kind": -1}, B.ERR_TYPE),
    ({"K": 0}, B.ERR_SHAPE), ({"K": 384}, B.ERR_SHAPE), ({"kind": B.Q4_0, "K": 48}, B.ERR_SHAPE),
    ({"K": 1 << 25, "ldo": 1 << 25}, B.ERR_SHAPE), ({"vocab": 0}, B.ERR_SHAPE), ({"vocab": 1 << 31}, B.ERR_SHAPE),
    ({"n": -1}, B.ERR_SHAPE), ({"n": 1 << 32}, B.ERR_SHAPE), ({"ldo": 511}, B.ERR_SHAPE),
    ({"table": P + 8}, B.ERR_ALIGN), ({"ids": ODD}, B.ERR_ALIGN), ({"out": ODD}, B.ERR_ALIGN),
    ({"n": 0}, 0), ({"n": 0, "table": None, "ids": None, "out": None}, 0), ({"kind": B.BF16, "K": 7, "n": 0}, 0),
])
def test_embed_refusals(L, kw, code):
    a = {**EMBED, **kw}
    assert L.mmvq_embed(*[a[k] for k in EMBED], None) == code


POOL = dict(page_table=P, pages_held=P, free_pages=P, n_free=P, pages_per_seq=8, n_pages=20, page_size=16)
PLAN = dict(cached=P, new=P, n_seqs=2, n_rows=5, start=P, length=P, seq=P, pos=P, slot=P, missing=P, ws=P, size=1 << 20)

BAD_POOL = [
    ({"page_table": None}, B.ERR_NULL), ({"pages_held": None}, B.ERR_NULL), ({"free_pages": None}, B.ERR_NULL),
    ({"n_free": None}, B.ERR_NULL), ({"pages_per_seq": 0}, B.ERR_SHAPE), ({"pages_per_seq": (1 << 26) + 1}, B.ERR_SHAPE),
    ({"table_stride": 7}, B.ERR_SHAPE), ({"n_pages": 0}, B.ERR_SHAPE), ({"page_size": 8}, B.ERR_SHAPE),
    ({"page_size": 24}, B.ERR_SHAPE), ({"page_size": 2048}, B.ERR_SHAPE),
    *[({k: ODD}, B.ERR_ALIGN) for k in ("page_table", "pages_held", "free_pages", "n_free")],
]


@pytest.mark.parametrize("kw,code", BAD_POOL)
def test_pool_refusals(L, kw, code):
    pool = B.kv_pool(**{**POOL, **kw})
    assert L.mmvq_kv_plan(pool, *PLAN.values(), None) == code
    assert L.mmvq_kv_release(pool, 2, P, None, None) == code


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, B.ERR_NULL) for k in ("cached", "new", "start", "length", "ws")],
    *[({k: ODD}, B.ERR_ALIGN) for k in ("cached", "new", "start", "length", "seq", "pos", "missing")],
    ({"slot": P + 4}, B.ERR_ALIGN), ({"ws": P + 8}, B.ERR_ALIGN), ({"n_seqs": -1}, B.ERR_SHAPE),
    ({"n_seqs": (1 << 20) + 1}, B.ERR_SHAPE), ({"n_rows": -1}, B.ERR_SHAPE), ({"n_rows": (1 << 20) + 1}, B.ERR_SHAPE),
    ({"size": 47}, B.ERR_SHAPE),
])
def test_plan_refusals(L, kw, code):
    assert L.mmvq_kv_plan(B.kv_pool(**POOL), *{**PLAN, **kw}.values(), None) == code
    assert L.mmvq_kv_plan(None, *PLAN.values(), None) == B.ERR_NULL


def test_release_refusals(L):
    pool = B.kv_pool(**POOL)
    assert L.mmvq_kv_release(None, 2, P, None, None) == B.ERR_NULL
    assert L.mmvq_kv_release(pool, 2, None, None, None) == B.ERR_NULL
    assert L.mmvq_kv_release(pool, 2, ODD, None, None) == B.ERR_ALIGN
    assert L.mmvq_kv_release(pool, 2, P, ODD, None) == B.ERR_ALIGN
    assert L.mmvq_kv_release(pool, -1, P, None, None) == B.ERR_SHAPE
    assert L.mmvq_kv_release(pool, (1 << 20) + 1, P, None, None) == B.ERR_SHAPE
    assert L.mmvq_kv_release(B.kv_pool(**{**POOL, "page_table": None, "pages_held": None}), 0, None, None, None) == 0


def test_plan_workspace(L):
    # 8 bytes of running sum and 4 of pages held a request, three numbers more
    assert B.mmvq_kv_plan_workspace(0) == 32 and B.mmvq_kv_plan_workspace(2) == 48
    assert B.mmvq_kv_plan_workspace(1 << 20) == 12 * (1 << 20) + 32
    assert L.mmvq_kv_plan_workspace(1, None) == B.ERR_NULL
    for bad in (-1, (1 << 20) + 1):
        with pytest.raises(B.MMVQError) as e:
            B.mmvq_kv_plan_workspace(bad)
        assert e.value.code == B.ERR_SHAPE


SET = dict(A=P, B=P, wtype=B.F16, n_adapters=3, K=64, M=50, max_rank=16, rank=P, scale=P)
LORA = dict(x=P, ldx=64, n=4, seq=P, adapter=P, n_seqs=2, base=P, ldb=50, out=P, ldo=50, ws=P, size=1 << 24)


@pytest.mark.parametrize("kw,code", [
    ({"wtype": B.Q4_0}, B.ERR_TYPE), ({"wtype": -1}, B.ERR_TYPE), ({"K": 60}, B.ERR_SHAPE), ({"K": 0}, B.ERR_SHAPE),
    ({"K": (1 << 20) + 8}, B.ERR_SHAPE), ({"M": 0}, B.ERR_SHAPE), ({"M": (1 << 24) + 1}, B.ERR_SHAPE),
    ({"max_rank": 0}, B.ERR_SHAPE), ({"max_rank": 12}, B.ERR_SHAPE), ({"max_rank": 264}, B.ERR_SHAPE),
    ({"n_adapters": 0}, B.ERR_SHAPE), ({"n_adapters": (1 << 20) + 1}, B.ERR_SHAPE), ({"stride_a": 16 * 64 - 8}, B.ERR_SHAPE),
    ({"stride_a": 16 * 64 + 4}, B.ERR_SHAPE), ({"stride_b": 50 * 16 - 8}, B.ERR_SHAPE), ({"stride_b": 50 * 16 + 4}, B.ERR_SHAPE),
])
def test_adapter_set_refusals(L, kw, code):
    s = B.lora_set(**{**SET, **kw})
    n = ctypes.c_int64()
    assert L.mmvq_lora_workspace(s, 4, n) == code
    assert L.mmvq_lora(s, P, 1 << 21, 4, P, P, 2, P, 1 << 25, P, 1 << 25, P, 1 << 40, None) == code


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, B.ERR_NULL) for k in ("x", "adapter", "base", "out", "ws")],
    *[({k: ODD}, B.ERR_ALIGN) for k in ("x", "seq", "adapter", "base", "out")], ({"ws": P + 8}, B.ERR_ALIGN),
    ({"ldx": 63}, B.ERR_SHAPE), ({"ldb": 49}, B.ERR_SHAPE), ({"ldo": 49}, B.ERR_SHAPE), ({"n": -1}, B.ERR_SHAPE),
    ({"n": (1 << 20) + 1}, B.ERR_SHAPE), ({"n_seqs": -1}, B.ERR_SHAPE), ({"seq": None}, B.ERR_SHAPE), ({"size": 255}, B.ERR_SHAPE),
    ({"ldb": 51}, B.ERR_SHAPE),                       # base is out, with another stride
    ({"n": 0}, 0), ({"n": 0, "x": None, "base": None, "out": None, "ws": None, "size": 0, "seq": None, "adapter": None}, 0),
])
def test_lora_refusals(L, kw, code):
    assert L.mmvq_lora(B.lora_set(**SET), *{**LORA, **kw}.values(), None) == code


def test_lora_set_pointers(L):
    for kw, code in [({"A": None}, B.ERR_NULL), ({"B": None}, B.ERR_NULL), ({"A": P + 8}, B.ERR_ALIGN), ({"B": P + 8}, B.ERR_ALIGN),
                     ({"rank": ODD}, B.ERR_ALIGN), ({"scale": ODD}, B.ERR_ALIGN)]:
        assert L.mmvq_lora(B.lora_set(**{**SET, **kw}), *LORA.values(), None) == code
    assert L.mmvq_lora(None, *LORA.values(), None) == B.ERR_NULL
    n = ctypes.c_int64()
    assert L.mmvq_lora_workspace(None, 1, n) == B.ERR_NULL
    assert L.mmvq_lora_workspace(B.lora_set(**SET), 1, None) == B.ERR_NULL
    assert L.mmvq_lora_workspace(B.lora_set(**SET), -1, n) == B.ERR_SHAPE
    assert B.mmvq_lora_workspace(B.lora_set(**SET), 0) == 0 and B.mmvq_lora_workspace(B.lora_set(**SET), 4) == 4 * 16 * 4


SAMPLE = dict(logits=P, ldl=100, vocab=100, n_rows=4, params=None, seq=P, n_seqs=2, u=P, tokens=P, chosen=P, probs=P + 4096, ldp=100,
              ws=P, size=1 << 24)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, B.ERR_NULL) for k in ("logits", "u", "ws")], ({"tokens": None, "chosen": None, "probs": None}, B.ERR_NULL),
    *[({k: ODD}, B.ERR_ALIGN) for k in ("logits", "seq", "u", "tokens", "chosen", "probs")], ({"ws": P + 8}, B.ERR_ALIGN),
    ({"ldl": 99}, B.ERR_SHAPE), ({"ldp": 99}, B.ERR_SHAPE), ({"vocab": 0}, B.ERR_SHAPE),
    ({"vocab": (1 << 24) + 1, "ldl": 1 << 25, "ldp": 1 << 25}, B.ERR_SHAPE), ({"n_rows": -1}, B.ERR_SHAPE),
    ({"n_rows": (1 << 20) + 1}, B.ERR_SHAPE), ({"n_seqs": -1}, B.ERR_SHAPE), ({"seq": None}, B.ERR_SHAPE), ({"size": 100}, B.ERR_SHAPE),
    ({"probs": P, "ldp": 101}, B.ERR_SHAPE),          # probs is logits, with another stride
    ({"n_rows": 0}, 0), ({"n_rows": 0, "logits": None, "u": None, "tokens": None, "chosen": None, "probs": None, "ws": None}, 0),
])
def test_sample_refusals(L, kw, code):
    assert L.mmvq_sample(*{**SAMPLE, **kw}.values(), None) == code


def test_sample_settings_and_workspace(L):
    for k in ("temperature", "top_k", "top_p", "min_p"):
        assert L.mmvq_sample(*{**SAMPLE, "params": B.sampling(**{k: ODD})}.values(), None) == B.ERR_ALIGN
    assert L.mmvq_sample_workspace(1, 1, None) == B.ERR_NULL
    for bad in ((-1, 1), (1, 0), (1, (1 << 24) + 1), ((1 << 20) + 1, 1)):
        with pytest.raises(B.MMVQError) as e:
            B.mmvq_sample_workspace(*bad)
        assert e.value.code == B.ERR_SHAPE
    assert B.mmvq_sample_workspace(0, 10) >= 0


def test_descriptors_keep_their_tensors():
    import torch
    for make, n in ((lambda t: B.kv_pool(*t, 1, 1, 16), 4), (lambda t: B.lora_set(t[0], t[1], B.F16, 1, 8, 1, 8, t[2], t[3]), 4),
                    (lambda t: B.sampling(*t), 4)):
        parts = [torch.zeros(4, dtype=torch.int32) for _ in range(n)]
        refs = [weakref.ref(x) for x in parts]
        made = make(parts)
        del parts
        gc.collect()
        assert all(r() is not None for r in refs)
        del made
        gc.collect()
        assert all(r() is None for r in refs)


def test_launch_arithmetic(tmp_path):
    """Rows, ranges of K and slices of M of an adapters' launch, over sizes up to the limits."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    clang = next((c for c in ("/opt/rocm/llvm/bin/clang++", shutil.which("clang++")) if c and os.path.exists(c)), None)
    if clang is None:
        pytest.skip("clang++ (host) not available")
    exe = tmp_path / "serve"
    subprocess.check_call([clang, "-std=c++17", "-O2", "-Wall", "-DQMV_HOST_MODEL", "-I",
                           os.path.join(root, "quantized_decode_gemv_quantize_amd", "csrc"), "-o", str(exe),
                           os.path.join(root, "tests", "host_model", "serve.cpp")])
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout[-4000:]
    assert "0 failing check(s)" in res.stdout
