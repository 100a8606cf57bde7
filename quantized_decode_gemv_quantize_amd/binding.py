"""Python binding of ``libmmvq.so`` (C ABI in ``include/mmvq.h``, for the
operators between the mat-vecs ``include/mmvq_decode.h`` and for those of a step
over many requests ``include/mmvq_serve.h``).

Argument marshalling only: every step of the computation runs in the HIP
library. Functions keep the C names; device buffers may be given as torch
tensors (their ``data_ptr()`` is passed) or as raw integer addresses, and
``stream`` as a torch stream, a raw ``hipStream_t`` integer, or ``None`` for
torch's current stream. A non-zero return code raises ``MMVQError``.

There is no fallback: if the library has not been built, loading raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB = os.path.join(HERE, "libmmvq.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "mmvq.h")
DECODE_HEADER = os.path.join(os.path.dirname(HERE), "include", "mmvq_decode.h")
SERVE_HEADER = os.path.join(os.path.dirname(HERE), "include", "mmvq_serve.h")

Q4_0, Q8_0, Q8_1, Q4_K, Q6_K = 2, 8, 9, 12, 14
Q4_1, Q5_0, Q5_1, Q5_K = 3, 6, 7, 13
F32, F16, BF16 = 0, 1, 30
TARGET_LOGITS, TARGET_WEIGHTS = 0, 1
GLU_PLAIN, GLU_SWIGLU, GLU_GEGLU, GLU_SWIGLU_OAI, GLU_SWIGLU_CLAMP = 0, 1, 2, 3, 4
MAX_COLS = 8
BLOCK = {Q4_0: (32, 18), Q8_0: (32, 34), Q4_K: (256, 144), Q6_K: (256, 210), Q8_1: (32, 36)}
DOTS_PER_BLOCK = {Q4_0: 1, Q8_0: 1, Q4_K: 16, Q6_K: 16}

ERR_NULL, ERR_TYPE, ERR_SHAPE, ERR_ALIGN, ERR_LAUNCH = -1, -2, -3, -4, -5

_i64 = ctypes.c_int64
_int = ctypes.c_int
_p = ctypes.c_void_p

class Epilogue(ctypes.Structure):
    """``mmvq_epilogue``: device pointers (ints, tensors via ``epilogue()``)."""
    _fields_ = [("up_bias", _p), ("gate_bias", _p), ("up_scale", _p), ("gate_scale", _p),
                ("glu_op", _int), ("glu_limit", ctypes.c_float)]


def epilogue(up_bias=None, gate_bias=None, up_scale=None, gate_scale=None, glu_op: int = 0,
             glu_limit: float = 0.0) -> Epilogue:
    e = Epilogue()
    e.up_bias, e.gate_bias = _addr(up_bias), _addr(gate_bias)
    e.up_scale, e.gate_scale = _addr(up_scale), _addr(gate_scale)
    e.glu_op, e.glu_limit = glu_op, glu_limit
    return e


_EP = ctypes.POINTER(Epilogue)


class KVCache(ctypes.Structure):
    """``mmvq_kv_cache``: addresses; made by ``kv_cache()`` it keeps the tensors, too."""
    _fields_ = [("k", _p), ("v", _p), ("type", _int), ("n_pages", _int), ("page_size", _int),
                ("n_kv_heads", _int), ("head_dim", _int)]


class KVBatch(ctypes.Structure):
    """``mmvq_kv_batch``: addresses; made by ``kv_batch()`` it keeps the tensors, too."""
    _fields_ = [("token_start", _p), ("seq_len", _p), ("page_table", _p), ("table_stride", _i64),
                ("n_seqs", _int), ("n_tokens", _int), ("pages_per_seq", _int), ("max_new", _int),
                ("max_len", _int)]


def kv_cache(k, v, kv_type: int, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int) -> KVCache:
    c = KVCache(_addr(k), _addr(v), kv_type, n_pages, page_size, n_kv_heads, head_dim)
    c.tensors = k, v
    return c


def kv_batch(token_start, seq_len, page_table, n_seqs: int, n_tokens: int, max_new: int, max_len: int,
             pages_per_seq: int, table_stride: int | None = None) -> KVBatch:
    b = KVBatch(_addr(token_start), _addr(seq_len), _addr(page_table),
                pages_per_seq if table_stride is None else table_stride, n_seqs, n_tokens, pages_per_seq,
                max_new, max_len)
    b.tensors = token_start, seq_len, page_table
    return b


class KVPool(ctypes.Structure):
    """``mmvq_kv_pool``: addresses; made by ``kv_pool()`` it keeps the tensors, too."""
    _fields_ = [("page_table", _p), ("table_stride", _i64), ("pages_held", _p), ("free_pages", _p), ("n_free", _p),
                ("pages_per_seq", _int), ("n_pages", _int), ("page_size", _int)]


class LoraSet(ctypes.Structure):
    """``mmvq_lora_set``: addresses; made by ``lora_set()`` it keeps the tensors, too."""
    _fields_ = [("A", _p), ("B", _p), ("rank", _p), ("scale", _p), ("stride_a", _i64), ("stride_b", _i64), ("K", _i64),
                ("M", _i64), ("type", _int), ("n_adapters", _int), ("max_rank", _int)]


class Sampling(ctypes.Structure):
    """``mmvq_sampling``: addresses; made by ``sampling()`` it keeps the tensors, too."""
    _fields_ = [("temperature", _p), ("top_k", _p), ("top_p", _p), ("min_p", _p)]


def kv_pool(page_table, pages_held, free_pages, n_free, pages_per_seq: int, n_pages: int, page_size: int,
            table_stride: int | None = None) -> KVPool:
    p = KVPool(_addr(page_table), pages_per_seq if table_stride is None else table_stride, _addr(pages_held),
               _addr(free_pages), _addr(n_free), pages_per_seq, n_pages, page_size)
    p.tensors = page_table, pages_held, free_pages, n_free
    return p


def lora_set(A, B, wtype: int, n_adapters: int, K: int, M: int, max_rank: int, rank=None, scale=None,
             stride_a: int | None = None, stride_b: int | None = None) -> LoraSet:
    s = LoraSet(_addr(A), _addr(B), _addr(rank), _addr(scale), max_rank * K if stride_a is None else stride_a,
                M * max_rank if stride_b is None else stride_b, K, M, wtype, n_adapters, max_rank)
    s.tensors = A, B, rank, scale
    return s


def sampling(temperature=None, top_k=None, top_p=None, min_p=None) -> Sampling:
    s = Sampling(_addr(temperature), _addr(top_k), _addr(top_p), _addr(min_p))
    s.tensors = temperature, top_k, top_p, min_p
    return s


_KC, _KB, _KP = ctypes.POINTER(KVCache), ctypes.POINTER(KVBatch), ctypes.POINTER(KVPool)
_LS, _SA = ctypes.POINTER(LoraSet), ctypes.POINTER(Sampling)
_pi64 = ctypes.POINTER(_i64)
_f32 = ctypes.c_float

_SIGS = {
    "mmvq_type_info": (_int, [_int, ctypes.POINTER(_int), ctypes.POINTER(_int)]),
    "mmvq_many_columns_min": (_int, [_int, _int, _int, ctypes.POINTER(_int)]),
    "mmvq_quantize_q8_1": (_int, [_p, _i64, _i64, _i64, _p, _p]),
    "mmvq": (_int, [_p, _int, _i64, _i64, _p, _i64, _p, _p]),
    "mmvq_glu": (_int, [_p, _p, _int, _i64, _i64, _p, _i64, _int, _p, _p]),
    "mmvq_id": (_int, [_p, _i64, _int, _int, _i64, _i64, _p, _i64, _p, _int, _p, _p]),
    "mmvq_id_glu": (_int, [_p, _p, _i64, _int, _int, _i64, _i64, _p, _i64, _p, _int, _int, _p, _p]),
    "mmvq_f32": (_int, [_p, _int, _i64, _i64, _p, _i64, _i64, _p, _p]),
    "mmvq_glu_f32": (_int, [_p, _p, _int, _i64, _i64, _p, _i64, _i64, _int, _p, _p]),
    "mmvq_id_f32": (_int, [_p, _i64, _int, _int, _i64, _i64, _p, _i64, _i64, _p, _int, _p, _p]),
    "mmvq_id_glu_f32": (_int, [_p, _p, _i64, _int, _int, _i64, _i64, _p, _i64, _i64, _p, _int, _int,
                               _p, _p]),
    "mmvq_ex": (_int, [_p, _p, _int, _i64, _i64, _p, _p, _i64, _i64, _EP, _p, _p]),
    "mmvq_id_ex": (_int, [_p, _p, _i64, _int, _int, _i64, _i64, _p, _p, _i64, _i64, _p, _int, _EP,
                          _p, _p, _p, _p, _p]),
    "mmvq_block_dots": (_int, [_p, _int, _i64, _i64, _p, _i64, _p, _p]),
    "mmvq_read_probe": (_int, [_p, _i64, _p, _p]),
    "mmvq_strerror": (ctypes.c_char_p, [_int]),
    "mmvq_add_rms_norm": (_int, [_p, _i64, _i64, _i64, _p, _i64, _p, _f32, _p, _i64, _p, _i64, _p, _p]),
    "mmvq_dequantize_q8_1": (_int, [_p, _i64, _i64, _p, _i64, _p]),
    "mmvq_kv_page_bytes": (_int, [_int, _int, _int, _int, _pi64]),
    "mmvq_kv_write": (_int, [_KC, _KB, _p, _i64, _p, _i64, _p]),
    "mmvq_kv_read": (_int, [_KC, _KB, _p, _i64, _p, _i64, _p]),
    "mmvq_attn_workspace": (_int, [_KC, _KB, _int, _pi64]),
    "mmvq_attn": (_int, [_KC, _KB, _p, _i64, _int, _f32, _int, _p, _p, _i64, _p, _i64, _p]),
    "mmvq_verify_workspace": (_int, [_int, _int, _int, _pi64]),
    "mmvq_verify_draft": (_int, [_p, _i64, _int, _int, _p, _p, _p, _i64, _p, _int, _int, _p, _p, _p, _p, _int,
                                 _p, _i64, _p]),
    "mmvq_embed": (_int, [_p, _int, _i64, _i64, _p, _i64, _f32, _p, _i64, _p]),
    "mmvq_kv_release": (_int, [_KP, _int, _p, _p, _p]),
    "mmvq_kv_plan_workspace": (_int, [_int, _pi64]),
    "mmvq_kv_plan": (_int, [_KP, _p, _p, _int, _int, _p, _p, _p, _p, _p, _p, _p, _i64, _p]),
    "mmvq_lora_workspace": (_int, [_LS, _i64, _pi64]),
    "mmvq_lora": (_int, [_LS, _p, _i64, _i64, _p, _p, _int, _p, _i64, _p, _i64, _p, _i64, _p]),
    "mmvq_sample_workspace": (_int, [_int, _int, _pi64]),
    "mmvq_sample": (_int, [_p, _i64, _int, _int, _SA, _p, _int, _p, _p, _p, _p, _i64, _p, _i64, _p]),
}

_lib = None


class MMVQError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {code}: {mmvq_strerror(code)}")
        self.code = code


def _load_hip() -> None:
    """torch's own HIP runtime, where torch is installed and no runtime is loaded yet: the library would bind
    to the system's, and torch bring its own beside it, on whose streams the library's launches fail."""
    with open("/proc/self/maps") as maps:
        if "libamdhip64" in maps.read():
            return
    spec = importlib.util.find_spec("torch")
    for where in (spec and spec.submodule_search_locations) or ():
        hip = os.path.join(where, "lib", "libamdhip64.so")
        if os.path.exists(hip):
            ctypes.CDLL(hip)
            return


def lib() -> ctypes.CDLL:
    """The loaded HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(f"{LIB} is missing: build it with "
                               "`python -m quantized_decode_gemv_quantize_amd.build`")
        _load_hip()
        L = ctypes.CDLL(LIB)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def declared_symbols(header: str = HEADER) -> list[str]:
    """Function names declared in include/mmvq.h."""
    text = open(header).read()
    return re.findall(r"^\s*(?:int|const char \*)\s*(mmvq\w*)\s*\(", text, flags=re.M)


def _addr(x) -> int | None:
    if x is None or x.__class__ is int:
        return x
    try:
        return x.data_ptr()
    except AttributeError:
        if isinstance(x, int):              # of a class of its own: rare, and the test costs every tensor
            return x
        raise


_torch = _current_device = _raw_stream = None


def _cuda():
    """torch, bound at the first launch, and its current device and current stream as plain numbers: without
    the check and the Stream object of torch.cuda's own functions where torch offers that (0.1 us for the two
    against 3), and without an import statement, which costs every call 0.2."""
    global _torch, _current_device, _raw_stream
    if _torch is None:
        import torch
        torch.cuda.init()
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
        _torch = torch
    return _torch


def _stream(s) -> int | None:
    if s is None:
        _cuda()
        return _raw_stream(_current_device())
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(fn: str, rc: int) -> int:
    if rc != 0:
        raise MMVQError(fn, rc)
    return rc


def mmvq_strerror(code: int) -> str:
    return lib().mmvq_strerror(code).decode()


def mmvq_type_info(wtype: int) -> tuple[int, int]:
    e, b = _int(), _int()
    _check("mmvq_type_info", lib().mmvq_type_info(wtype, ctypes.byref(e), ctypes.byref(b)))
    return e.value, b.value


def mmvq_many_columns_min(wtype: int, gated: bool, fp32: bool = False) -> int:
    n = _int()
    _check("mmvq_many_columns_min",
           lib().mmvq_many_columns_min(wtype, int(bool(gated)), int(bool(fp32)), ctypes.byref(n)))
    return n.value


def mmvq_quantize_q8_1(x, K: int, n: int, ldx: int, y_q, stream=None) -> None:
    _check("mmvq_quantize_q8_1",
           lib().mmvq_quantize_q8_1(_addr(x), K, n, ldx, _addr(y_q), _stream(stream)))


def mmvq(W, wtype: int, M: int, K: int, y_q, n: int, out, stream=None) -> None:
    _check("mmvq", lib().mmvq(_addr(W), wtype, M, K, _addr(y_q), n, _addr(out), _stream(stream)))


def mmvq_glu(W_gate, W_up, wtype: int, M: int, K: int, y_q, n: int, glu_op: int, out,
             stream=None) -> None:
    _check("mmvq_glu", lib().mmvq_glu(_addr(W_gate), _addr(W_up), wtype, M, K, _addr(y_q), n,
                                      glu_op, _addr(out), _stream(stream)))


def mmvq_id(W, expert_stride_bytes: int, n_experts: int, wtype: int, M: int, K: int, y_q,
            n_tokens: int, ids, top_k: int, out, stream=None) -> None:
    _check("mmvq_id", lib().mmvq_id(_addr(W), expert_stride_bytes, n_experts, wtype, M, K,
                                    _addr(y_q), n_tokens, _addr(ids), top_k, _addr(out),
                                    _stream(stream)))


def mmvq_id_glu(W_gate, W_up, expert_stride_bytes: int, n_experts: int, wtype: int, M: int,
                K: int, y_q, n_tokens: int, ids, top_k: int, glu_op: int, out,
                stream=None) -> None:
    _check("mmvq_id_glu", lib().mmvq_id_glu(_addr(W_gate), _addr(W_up), expert_stride_bytes,
                                            n_experts, wtype, M, K, _addr(y_q), n_tokens,
                                            _addr(ids), top_k, glu_op, _addr(out),
                                            _stream(stream)))


def mmvq_f32(W, wtype: int, M: int, K: int, x, n: int, ldx: int, out, stream=None) -> None:
    _check("mmvq_f32", lib().mmvq_f32(_addr(W), wtype, M, K, _addr(x), n, ldx, _addr(out),
                                      _stream(stream)))


def mmvq_glu_f32(W_gate, W_up, wtype: int, M: int, K: int, x, n: int, ldx: int, glu_op: int,
                 out, stream=None) -> None:
    _check("mmvq_glu_f32", lib().mmvq_glu_f32(_addr(W_gate), _addr(W_up), wtype, M, K, _addr(x),
                                              n, ldx, glu_op, _addr(out), _stream(stream)))


def mmvq_id_f32(W, expert_stride_bytes: int, n_experts: int, wtype: int, M: int, K: int, x,
                n_tokens: int, ldx: int, ids, top_k: int, out, stream=None) -> None:
    _check("mmvq_id_f32", lib().mmvq_id_f32(_addr(W), expert_stride_bytes, n_experts, wtype, M, K,
                                            _addr(x), n_tokens, ldx, _addr(ids), top_k,
                                            _addr(out), _stream(stream)))


def mmvq_id_glu_f32(W_gate, W_up, expert_stride_bytes: int, n_experts: int, wtype: int, M: int,
                    K: int, x, n_tokens: int, ldx: int, ids, top_k: int, glu_op: int, out,
                    stream=None) -> None:
    _check("mmvq_id_glu_f32", lib().mmvq_id_glu_f32(_addr(W_gate), _addr(W_up),
                                                    expert_stride_bytes, n_experts, wtype, M, K,
                                                    _addr(x), n_tokens, ldx, _addr(ids), top_k,
                                                    glu_op, _addr(out), _stream(stream)))


def _ep(epi):
    return None if epi is None else ctypes.byref(epi)


def mmvq_ex(W_up, W_gate, wtype: int, M: int, K: int, y_q, x, ldx: int, n: int,
            epi: Epilogue | None, out, stream=None) -> None:
    _check("mmvq_ex", lib().mmvq_ex(_addr(W_up), _addr(W_gate), wtype, M, K, _addr(y_q), _addr(x), ldx,
                                    n, _ep(epi), _addr(out), _stream(stream)))


def mmvq_id_ex(W_up, W_gate, expert_stride_bytes: int, n_experts: int, wtype: int, M: int, K: int,
               y_q, x, ldx: int, n_tokens: int, ids, top_k: int, epi: Epilogue | None,
               shared_up, shared_gate, shared_out, out, stream=None) -> None:
    _check("mmvq_id_ex", lib().mmvq_id_ex(_addr(W_up), _addr(W_gate), expert_stride_bytes, n_experts,
                                          wtype, M, K, _addr(y_q), _addr(x), ldx, n_tokens, _addr(ids),
                                          top_k, _ep(epi), _addr(shared_up), _addr(shared_gate),
                                          _addr(shared_out), _addr(out), _stream(stream)))


def mmvq_block_dots(W, wtype: int, M: int, K: int, y_q, n: int, dots, stream=None) -> None:
    _check("mmvq_block_dots", lib().mmvq_block_dots(_addr(W), wtype, M, K, _addr(y_q), n,
                                                    _addr(dots), _stream(stream)))


# ---------------------------------------------------------------------------
# Operators between the mat-vecs (include/mmvq_decode.h)
# ---------------------------------------------------------------------------

def _launch(fn: str, where, stream, *args) -> None:
    """Calls ``fn`` on ``stream``; without one, on the current stream of the device of ``where``, which
    need not be the current device."""
    f = getattr(_lib or lib(), fn)
    if stream is not None:
        handle = _stream(stream)
        index = None if handle else getattr(stream, "device_index", None)
        if index is None:
            rc = f(*args, handle)
        else:                               # a device's default stream: the handle does not say of which
            with (_torch or _cuda()).cuda.device(index):
                rc = f(*args, handle)
    else:
        torch = _torch or _cuda()
        here = _current_device()
        index = here if where is None or isinstance(where, int) else where.get_device()
        if index == here or index < 0:
            rc = f(*args, _raw_stream(here))
        else:
            with torch.cuda.device(index):
                rc = f(*args, _raw_stream(index))
    if rc:
        _check(fn, rc)


def mmvq_add_rms_norm(x, K: int, n: int, ldx: int, residual, ldr: int, weight, eps: float, sum_out, lds: int,
                      y, ldy: int, y_q, stream=None) -> None:
    _launch("mmvq_add_rms_norm", x, stream, _addr(x), K, n, ldx, _addr(residual), ldr, _addr(weight), eps,
            _addr(sum_out), lds, _addr(y), ldy, _addr(y_q))


def mmvq_dequantize_q8_1(y_q, K: int, n: int, x, ldx: int, stream=None) -> None:
    _launch("mmvq_dequantize_q8_1", x, stream, _addr(y_q), K, n, _addr(x), ldx)


def mmvq_kv_page_bytes(kv_type: int, page_size: int, n_kv_heads: int, head_dim: int) -> int:
    n = _i64()
    _check("mmvq_kv_page_bytes", lib().mmvq_kv_page_bytes(kv_type, page_size, n_kv_heads, head_dim, n))
    return n.value


def mmvq_kv_write(cache: KVCache, batch: KVBatch, k, ldk: int, v, ldv: int, stream=None) -> None:
    _launch("mmvq_kv_write", k, stream, cache, batch, _addr(k), ldk, _addr(v), ldv)


def mmvq_kv_read(cache: KVCache, batch: KVBatch, k, ldk: int, v, ldv: int, stream=None) -> None:
    _launch("mmvq_kv_read", v if k is None else k, stream, cache, batch, _addr(k), ldk, _addr(v), ldv)


def mmvq_attn_workspace(cache: KVCache, batch: KVBatch, n_heads: int) -> int:
    n = _i64()
    _check("mmvq_attn_workspace", lib().mmvq_attn_workspace(cache, batch, n_heads, n))
    return n.value


def mmvq_attn(cache: KVCache, batch: KVBatch, q, ldq: int, n_heads: int, scale: float, window: int, sinks, out,
              ldo: int, workspace, workspace_bytes: int, stream=None) -> None:
    _launch("mmvq_attn", q, stream, cache, batch, _addr(q), ldq, n_heads, scale, window, _addr(sinks),
            _addr(out), ldo, _addr(workspace), workspace_bytes)


def mmvq_verify_workspace(n_seqs: int, n_rows: int, vocab: int) -> int:
    n = _i64()
    _check("mmvq_verify_workspace", lib().mmvq_verify_workspace(n_seqs, n_rows, vocab, n))
    return n.value


def mmvq_verify_draft(target, ldt: int, vocab: int, kind: int, temperature, draft_tokens, draft_probs, ldd: int,
                      row_start, n_seqs: int, n_rows: int, u_accept, u_sample, n_accepted, tokens, max_out: int,
                      workspace, workspace_bytes: int, stream=None) -> None:
    _launch("mmvq_verify_draft", target, stream, _addr(target), ldt, vocab, kind, _addr(temperature),
            _addr(draft_tokens), _addr(draft_probs), ldd, _addr(row_start), n_seqs, n_rows, _addr(u_accept),
            _addr(u_sample), _addr(n_accepted), _addr(tokens), max_out, _addr(workspace), workspace_bytes)


# ---------------------------------------------------------------------------
# Operators of a step over many requests (include/mmvq_serve.h)
# ---------------------------------------------------------------------------

def mmvq_embed(table, wtype: int, vocab: int, K: int, ids, n: int, scale: float, out, ldo: int, stream=None) -> None:
    _launch("mmvq_embed", out, stream, _addr(table), wtype, vocab, K, _addr(ids), n, scale, _addr(out), ldo)


def mmvq_kv_release(pool: KVPool, n_seqs: int, keep, shared=None, stream=None) -> None:
    _launch("mmvq_kv_release", keep, stream, pool, n_seqs, _addr(keep), _addr(shared))


def mmvq_kv_plan_workspace(n_seqs: int) -> int:
    n = _i64()
    _check("mmvq_kv_plan_workspace", lib().mmvq_kv_plan_workspace(n_seqs, n))
    return n.value


def mmvq_kv_plan(pool: KVPool, cached, n_new, n_seqs: int, n_rows: int, token_start, seq_len, row_seq, row_pos,
                 row_slot, n_missing, workspace, workspace_bytes: int, stream=None) -> None:
    _launch("mmvq_kv_plan", token_start, stream, pool, _addr(cached), _addr(n_new), n_seqs, n_rows,
            _addr(token_start), _addr(seq_len), _addr(row_seq), _addr(row_pos), _addr(row_slot), _addr(n_missing),
            _addr(workspace), workspace_bytes)


def mmvq_lora_workspace(adapters: LoraSet, n: int) -> int:
    b = _i64()
    _check("mmvq_lora_workspace", lib().mmvq_lora_workspace(adapters, n, b))
    return b.value


def mmvq_lora(adapters: LoraSet, x, ldx: int, n: int, row_seq, adapter, n_seqs: int, base, ldb: int, out, ldo: int,
              workspace, workspace_bytes: int, stream=None) -> None:
    _launch("mmvq_lora", x, stream, adapters, _addr(x), ldx, n, _addr(row_seq), _addr(adapter), n_seqs, _addr(base),
            ldb, _addr(out), ldo, _addr(workspace), workspace_bytes)


def mmvq_sample_workspace(n_rows: int, vocab: int) -> int:
    n = _i64()
    _check("mmvq_sample_workspace", lib().mmvq_sample_workspace(n_rows, vocab, n))
    return n.value


def mmvq_sample(logits, ldl: int, vocab: int, n_rows: int, params: Sampling | None, row_seq, n_seqs: int, u, tokens,
                chosen, probs, ldp: int, workspace, workspace_bytes: int, stream=None) -> None:
    _launch("mmvq_sample", logits, stream, _addr(logits), ldl, vocab, n_rows, params, _addr(row_seq), n_seqs,
            _addr(u), _addr(tokens), _addr(chosen), _addr(probs), ldp, _addr(workspace), workspace_bytes)


# ---------------------------------------------------------------------------
# Tensor-level conveniences (allocate outputs with torch, then call the ABI)
# ---------------------------------------------------------------------------

def mmvq_read_probe(src, nbytes: int, sink, stream=None) -> None:
    _check("mmvq_read_probe", lib().mmvq_read_probe(_addr(src), nbytes, _addr(sink), _stream(stream)))


def quantize(x, K: int | None = None, stream=None):
    """x: float32 CUDA tensor [n, ldx] -> uint8 tensor [n, (K/32)*36]."""
    import torch
    if x.dim() == 1:
        x = x.view(1, -1)
    n, ldx = x.shape
    K = ldx if K is None else K
    y = torch.empty((n, K // 32 * 36), dtype=torch.uint8, device=x.device)
    mmvq_quantize_q8_1(x, K, n, x.stride(0), y, stream)
    return y


def gemv(W, wtype: int, M: int, K: int, y_q, n: int, stream=None):
    """-> float32 tensor [n, M]."""
    import torch
    out = torch.empty((n, M), dtype=torch.float32, device=y_q.device)
    mmvq(W, wtype, M, K, y_q, n, out, stream)
    return out
