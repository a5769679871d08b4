"""Python binding of the C ABI in ``include/ns_paged.h`` (argument marshalling only).

Every function here has the name of the C entry point it calls and does no
arithmetic of its own: it checks tensor shapes, takes device pointers and the
current CUDA stream from torch, calls the library and raises on a non-zero
status.  torch serves only as the allocator and stream provider.  There is
no CPU fallback: if ``_lib/libns_paged.so`` is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import _build

NS_OK = 0
NS_F16 = 0
NS_BF16 = 1
NS_MAX_CTAS = 1024
NS_PREFILL_WALK = 1
NS_PREFILL_TENSOR_CORE = 2
NS_NOALLOC_MAX_PAIRS = 16384
DEV_BITS = {
    0x1: "NS_DEV_BAD_BLOCK_ID",
    0x2: "NS_DEV_BAD_CONTEXT_LEN",
    0x4: "NS_DEV_BAD_SLOT",
    0x8: "NS_DEV_WAIT_TIMEOUT",
    0x10: "NS_DEV_FUSED_SLOT",
    0x20: "NS_DEV_BAD_QUERY_SPAN",
    0x40: "NS_DEV_MERGE_QUEUE",
    0x80: "NS_DEV_BAD_TOKEN",
}


class NsError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = lib().ns_status_string(status).decode()
        super().__init__(f"{what}: {msg} ({status})")


class DecodeConfig(ctypes.Structure):
    _fields_ = [("num_ctas", ctypes.c_int), ("min_blocks_per_cta", ctypes.c_int),
                ("whole_sequences", ctypes.c_int), ("overlap_prologue", ctypes.c_int),
                ("wait_limit_ns", ctypes.c_int), ("merge_levels", ctypes.c_int), ("reserved", ctypes.c_int * 2)]


class PrefillConfig(ctypes.Structure):
    _fields_ = [("tensor_core_min_span", ctypes.c_int), ("phases", ctypes.c_int),
                ("reserved", ctypes.c_int * 6)]


class DecodePlan(ctypes.Structure):
    _fields_ = [("ctas_launched", ctypes.c_int32), ("ctas_active", ctypes.c_int32),
                ("total_blocks", ctypes.c_int64), ("split_pairs", ctypes.c_int32),
                ("max_pieces", ctypes.c_int32), ("whole_sequences", ctypes.c_int32),
                ("workers_active", ctypes.c_int32), ("merge_levels", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 7)]


_LIB = None
P, I, I64, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t

_SIGNATURES = {
    "ns_status_string": (ctypes.c_char_p, [I]),
    "ns_version": (I, []),
    "ns_kv_append": (I, [P, P, P, P, P, I, I, I, I, I64, I, P]),
    "ns_paged_attn_workspace_bytes": (SZ, [I, I, I, I]),
    "ns_paged_attn_workspace_init": (I, [P, SZ, P]),
    "ns_paged_attn_decode": (I, [P, P, P, P, P, I, I, I, I, I, F, P, P, I, I64, I, P, SZ]),
    "ns_paged_attn_decode_ex": (I, [P, P, P, P, P, I, I, I, I, I, F, P, P, I, I64, I, P, SZ,
                                    ctypes.POINTER(DecodeConfig)]),
    "ns_kv_append_paged_attn_decode": (I, [P, P, P, P, P, P, P, P, I, I, I, I, I, F, P, P, I,
                                           I64, I, P, SZ]),
    "ns_kv_append_paged_attn_decode_ex": (I, [P, P, P, P, P, P, P, P, I, I, I, I, I, F, P, P, I,
                                              I64, I, P, SZ, ctypes.POINTER(DecodeConfig)]),
    "ns_read_decode_plan": (I, [P, ctypes.POINTER(DecodePlan), P]),
    "ns_paged_attn_prefill": (I, [P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, I, I64, I, P, SZ]),
    "ns_paged_attn_prefill_ex": (I, [P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, I, I64, I, P, SZ,
                                     ctypes.POINTER(PrefillConfig)]),
    "ns_get_device_status": (I, [P, ctypes.POINTER(ctypes.c_uint32), I]),
    "ns_paged_attn_decode_noalloc": (I, [P, P, P, P, P, I, I, I, I, I, F, P, P, I, I64, I]),
    "ns_kv_append_q8_0": (I, [P, P, P, P, P, P, P, I, I, I, I, I64, I, P]),
    "ns_paged_attn_decode_q8_0": (I, [P, P, P, P, P, P, P, I, I, I, I, I, F, P, P, I, I64, I, P, SZ]),
    "ns_kv_append_paged_attn_decode_q8_0": (I, [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, F, P, P, I,
                                                I64, I, P, SZ]),
    "ns_span_attn_workspace_bytes": (SZ, [I]),
    "ns_prompt_attn": (I, [P, P, P, P, P, I, I, I, I, I, I, I64, I64, I64, F, P, P, I, P, SZ]),
    "ns_paged_attn_prefill_q8_0": (I, [P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, I, I64, I, P, SZ]),
    "ns_kv_gather": (I, [P, P, P, P, I, I, I, I, I, P, P, P, I, I64, I]),
    "ns_kv_gather_q8_0": (I, [P, P, P, P, P, P, I, I, I, I, I, P, P, P, I, I64, I]),
    "ns_verify_drafts": (I, [P, P, P, P, P, P, I, I, I, I64, I64, P, P, P]),
}


def lib_path() -> str:
    return _build.LIB


def lib():
    """The loaded C library (raises if it was never built: there is no fallback)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(_build.LIB):
            raise RuntimeError(
                f"{_build.LIB} is missing: build it with __graft_entry__.build() "
                "(the paged-KV kernels have no CPU fallback)")
        handle = ctypes.CDLL(_build.LIB)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = handle
    return _LIB


def _check(status: int, what: str):
    if status != NS_OK:
        raise NsError(status, what)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return NS_F16
    if t.dtype == torch.bfloat16:
        return NS_BF16
    raise TypeError(f"expected float16 or bfloat16, got {t.dtype}")


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    try:
        if t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype is dtype):
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


# The current stream's handle without the Python object around it (3 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int:
    if _capture.on:
        return _STREAM_SLOT
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_raw_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# While a call is prepared, the entry points record their marshalled arguments
# instead of calling the library, and the stream argument is a slot filled in
# at each run.
class _Capture(threading.local):
    on = False
    record = None


_capture = _Capture()
_STREAM_SLOT = object()


def _invoke(name: str, *args) -> int:
    if _capture.on:
        _capture.record = (name, args)
        return NS_OK
    return getattr(_LIB or lib(), name)(*args)


class PreparedCall:
    """One launching entry point with its arguments checked and marshalled once.

    Calling it runs the same C entry point again on the same buffers (with
    whatever they hold then) on ``stream`` (default: the current stream); only
    the stream is looked up per call.  The object references every tensor and
    config it was prepared with, so their memory stays allocated while it
    lives.  One object must not be called from two threads at once.
    """

    __slots__ = ("name", "_fn", "_args", "_slot", "_keep")

    def __init__(self, name: str, args: tuple, keep: list):
        self.name = name
        self._fn = getattr(lib(), name)
        self._args = list(args)
        slots = [i for i, a in enumerate(self._args) if a is _STREAM_SLOT]
        if len(slots) != 1:
            raise RuntimeError(f"{name}: expected one stream argument")
        self._slot = slots[0]
        self._keep = keep

    def __call__(self, stream=None):
        self._args[self._slot] = _stream(stream)
        _check(self._fn(*self._args), self.name)


def prepare(fn, *args, **kwargs) -> PreparedCall:
    """``fn`` (a launching entry point of this module: ns_kv_append,
    ns_paged_attn_decode, ns_kv_append_paged_attn_decode, ns_paged_attn_prefill,
    a q8_0 one, ns_prompt_attn, ns_kv_gather or ns_verify_drafts) with these
    arguments, checked now and run by calling the returned object.  It is what a
    serving loop that calls the same step on the same buffers every iteration
    uses, so that a call costs the host one foreign call."""
    if kwargs.get("stream") is not None:
        raise ValueError("the stream is given to each run of a prepared call")
    _capture.on, _capture.record = True, None
    try:
        fn(*args, **kwargs)
    except ctypes.ArgumentError as e:  # an entry point that calls the library directly
        raise TypeError(f"{getattr(fn, '__name__', fn)} cannot be prepared") from e
    finally:
        _capture.on = False
    if _capture.record is None:
        raise TypeError(f"{getattr(fn, '__name__', fn)} cannot be prepared")
    name, marshalled = _capture.record
    _capture.record = None
    keep = [a for a in list(args) + list(kwargs.values()) if a is not None]
    return PreparedCall(name, marshalled, keep)


def ns_version() -> int:
    return lib().ns_version()


def ns_paged_attn_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                                  head_dim: int = 64) -> int:
    return int(lib().ns_paged_attn_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim))


def alloc_workspace(num_rows: int, num_q_heads: int, num_kv_heads: int, head_dim: int = 64,
                    device=None) -> torch.Tensor:
    """A zero-filled workspace for up to ``num_rows`` query rows (sequences when decoding)."""
    n = ns_paged_attn_workspace_bytes(num_rows, num_q_heads, num_kv_heads, head_dim)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def ns_kv_append(k, v, slot_mapping, k_pool, v_pool, stream=None):
    """Write k/v [T, Hkv, D] into k_pool/v_pool [NB, Hkv, bs, D] at slot_mapping [T] (int64)."""
    T, hkv, d = k.shape
    nb, hkv2, bs, d2 = k_pool.shape
    if v.shape != k.shape or v_pool.shape != k_pool.shape or hkv2 != hkv or d2 != d:
        raise ValueError("shape mismatch")
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [num_tokens]")
    dt = _dtype_code(k)
    st = _invoke("ns_kv_append", _dev(k, "k"), _dev(v, "v", k.dtype),
                 _dev(slot_mapping, "slot_mapping", torch.int64),
                 _dev(k_pool, "k_pool", k.dtype), _dev(v_pool, "v_pool", k.dtype),
                 T, hkv, d, bs, nb, dt, _stream(stream))
    _check(st, "ns_kv_append")


def _attn_common(q, k_pool, v_pool, block_tables, context_lens, out, workspace):
    rows, hq, d = q.shape
    nb, hkv, bs, d2 = k_pool.shape
    if v_pool.shape != k_pool.shape or d2 != d:
        raise ValueError("pool shapes do not match q")
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    dt = _dtype_code(q)
    ptrs = dict(q=_dev(q, "q"), k=_dev(k_pool, "k_pool", q.dtype), v=_dev(v_pool, "v_pool", q.dtype),
                bt=_dev(block_tables, "block_tables", torch.int32),
                cl=_dev(context_lens, "context_lens", torch.int32),
                out=_dev(out, "out", q.dtype), ws=_dev(workspace, "workspace", torch.uint8))
    return rows, hq, hkv, d, bs, nb, dt, ptrs


def ns_paged_attn_decode(q, k_pool, v_pool, block_tables, context_lens, scale, out, workspace,
                         config: DecodeConfig | None = None, stream=None):
    """out[s] = paged attention of q[s] over sequence s's blocks (one decode step)."""
    S, hq, hkv, d, bs, nb, dt, p = _attn_common(q, k_pool, v_pool, block_tables, context_lens,
                                                out, workspace)
    if context_lens.shape != (S,) or block_tables.shape[0] != S:
        raise ValueError("one context length and one table row per sequence")
    args = (p["q"], p["k"], p["v"], p["bt"], p["cl"], S, hq, hkv, d, bs, float(scale), p["out"],
            _stream(stream), block_tables.shape[1], nb, dt, p["ws"], workspace.numel())
    if config is None:
        _check(_invoke("ns_paged_attn_decode", *args), "ns_paged_attn_decode")
    else:
        _check(_invoke("ns_paged_attn_decode_ex", *args, ctypes.byref(config)), "ns_paged_attn_decode_ex")


def ns_paged_attn_decode_noalloc(q, k_pool, v_pool, block_tables, context_lens, scale, out,
                                 stream=None):
    """ns_paged_attn_decode for callers that cannot allocate device memory.

    Takes no workspace: the library's own scratch array holds the split
    partials and counters (at most NS_NOALLOC_MAX_PAIRS sequence x kv-head
    pairs).  The first call on a device must come before any stream capture;
    calls that overlap on the GPU race.
    """
    S, hq, d = q.shape
    nb_, hkv, bs, d2 = k_pool.shape
    if v_pool.shape != k_pool.shape or d2 != d or out.shape != q.shape:
        raise ValueError("shape mismatch")
    if context_lens.shape != (S,) or block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("one context length and one table row per sequence")
    st = lib().ns_paged_attn_decode_noalloc(
        _dev(q, "q"), _dev(k_pool, "k_pool", q.dtype), _dev(v_pool, "v_pool", q.dtype),
        _dev(block_tables, "block_tables", torch.int32),
        _dev(context_lens, "context_lens", torch.int32), S, hq, hkv, d, bs, float(scale),
        _dev(out, "out", q.dtype), _stream(stream), block_tables.shape[1], nb_, _dtype_code(q))
    _check(st, "ns_paged_attn_decode_noalloc")


def ns_kv_append_paged_attn_decode(q, k_new, v_new, slot_mapping, k_pool, v_pool, block_tables,
                                   context_lens, scale, out, workspace, config: DecodeConfig | None = None,
                                   stream=None):
    """Append one new token per sequence and run the decode step, in one kernel."""
    S, hq, hkv, d, bs, nb, dt, p = _attn_common(q, k_pool, v_pool, block_tables, context_lens,
                                                out, workspace)
    if k_new.shape != (S, hkv, d) or v_new.shape != (S, hkv, d) or slot_mapping.shape != (S,):
        raise ValueError("k_new/v_new must be [num_seqs, Hkv, D], slot_mapping [num_seqs]")
    st = _invoke(
        "ns_kv_append_paged_attn_decode_ex",
        p["q"], _dev(k_new, "k_new", q.dtype), _dev(v_new, "v_new", q.dtype),
        _dev(slot_mapping, "slot_mapping", torch.int64), p["k"], p["v"], p["bt"], p["cl"], S, hq,
        hkv, d, bs, float(scale), p["out"], _stream(stream), block_tables.shape[1], nb, dt,
        p["ws"], workspace.numel(), ctypes.byref(config) if config is not None else None)
    _check(st, "ns_kv_append_paged_attn_decode")


def ns_paged_attn_prefill(q, query_start_loc, k_pool, v_pool, block_tables, context_lens, scale,
                          out, workspace, config: PrefillConfig | None = None, stream=None):
    """Chunked-prefill attention of the query spans ``query_start_loc`` over the paged pool."""
    T, hq, hkv, d, bs, nb, dt, p = _attn_common(q, k_pool, v_pool, block_tables, context_lens,
                                                out, workspace)
    S = context_lens.shape[0]
    if query_start_loc.shape != (S + 1,) or block_tables.shape[0] != S:
        raise ValueError("query_start_loc must be [num_seqs + 1]")
    args = (p["q"], _dev(query_start_loc, "query_start_loc", torch.int32), p["k"], p["v"], p["bt"],
            p["cl"], S, T, hq, hkv, d, bs, float(scale), p["out"], _stream(stream),
            block_tables.shape[1], nb, dt, p["ws"], workspace.numel())
    if config is None:
        _check(_invoke("ns_paged_attn_prefill", *args), "ns_paged_attn_prefill")
    else:
        _check(_invoke("ns_paged_attn_prefill_ex", *args, ctypes.byref(config)),
               "ns_paged_attn_prefill_ex")


def _q8_pools(k_codes, k_scales, v_codes, v_scales):
    nb, hkv, bs, d = k_codes.shape
    if v_codes.shape != k_codes.shape or k_scales.shape != (nb, hkv, bs, d // 32) \
            or v_scales.shape != k_scales.shape:
        raise ValueError("q8_0 pools: codes [NB, Hkv, bs, D] int8, scales [NB, Hkv, bs, D/32] fp16")
    return (nb, hkv, bs, d, _dev(k_codes, "k_codes", torch.int8), _dev(k_scales, "k_scales", torch.float16),
            _dev(v_codes, "v_codes", torch.int8), _dev(v_scales, "v_scales", torch.float16))


def ns_kv_append_q8_0(k, v, slot_mapping, k_codes, k_scales, v_codes, v_scales, stream=None):
    """Quantise k/v [T, Hkv, D] to q8_0 and write codes and scales at slot_mapping [T] (int64)."""
    T, hkv, d = k.shape
    nb, hkv2, bs, d2, kc, ks, vc, vs = _q8_pools(k_codes, k_scales, v_codes, v_scales)
    if v.shape != k.shape or hkv2 != hkv or d2 != d or slot_mapping.shape != (T,):
        raise ValueError("shape mismatch")
    st = _invoke("ns_kv_append_q8_0", _dev(k, "k"), _dev(v, "v", k.dtype),
                 _dev(slot_mapping, "slot_mapping", torch.int64), kc, ks, vc, vs, T, hkv, d,
                 bs, nb, _dtype_code(k), _stream(stream))
    _check(st, "ns_kv_append_q8_0")


def ns_paged_attn_decode_q8_0(q, k_codes, k_scales, v_codes, v_scales, block_tables, context_lens, scale,
                              out, workspace, stream=None):
    """Decode attention of q [S, Hq, D] over a q8_0 pool (block size 16)."""
    S, hq, d = q.shape
    nb, hkv, bs, d2, kc, ks, vc, vs = _q8_pools(k_codes, k_scales, v_codes, v_scales)
    if d2 != d or out.shape != q.shape or context_lens.shape != (S,) or block_tables.shape[0] != S:
        raise ValueError("shape mismatch")
    st = _invoke(
        "ns_paged_attn_decode_q8_0",
        _dev(q, "q"), kc, ks, vc, vs, _dev(block_tables, "block_tables", torch.int32),
        _dev(context_lens, "context_lens", torch.int32), S, hq, hkv, d, bs, float(scale),
        _dev(out, "out", q.dtype), _stream(stream), block_tables.shape[1], nb, _dtype_code(q),
        _dev(workspace, "workspace", torch.uint8), workspace.numel())
    _check(st, "ns_paged_attn_decode_q8_0")


def ns_kv_append_paged_attn_decode_q8_0(q, k_new, v_new, slot_mapping, k_codes, k_scales, v_codes, v_scales,
                                        block_tables, context_lens, scale, out, workspace, stream=None):
    """Quantise and append one new token per sequence, then decode over the q8_0 pool, in one kernel."""
    S, hq, d = q.shape
    nb, hkv, bs, d2, kc, ks, vc, vs = _q8_pools(k_codes, k_scales, v_codes, v_scales)
    if k_new.shape != (S, hkv, d) or v_new.shape != (S, hkv, d) or slot_mapping.shape != (S,):
        raise ValueError("k_new/v_new must be [num_seqs, Hkv, D], slot_mapping [num_seqs]")
    if d2 != d or out.shape != q.shape or context_lens.shape != (S,) or block_tables.shape[0] != S:
        raise ValueError("shape mismatch")
    st = _invoke("ns_kv_append_paged_attn_decode_q8_0", 
        _dev(q, "q"), _dev(k_new, "k_new", q.dtype), _dev(v_new, "v_new", q.dtype),
        _dev(slot_mapping, "slot_mapping", torch.int64), kc, ks, vc, vs,
        _dev(block_tables, "block_tables", torch.int32), _dev(context_lens, "context_lens", torch.int32), S, hq,
        hkv, d, bs, float(scale), _dev(out, "out", q.dtype), _stream(stream), block_tables.shape[1], nb,
        _dtype_code(q), _dev(workspace, "workspace", torch.uint8), workspace.numel())
    _check(st, "ns_kv_append_paged_attn_decode_q8_0")


def _rows(t: torch.Tensor, name: str, dtype, shape):
    """Pointer of [T, H, D] rows that are dense themselves, and elements from one to the next
    (with no next row, the row's own width)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if n and h and d and ((s2 != 1 and d > 1) or (s1 != d and h > 1)):
        raise ValueError(f"the rows of {name} must be dense [heads, head_dim]")
    return t.data_ptr(), s0 if n > 1 else h * d


def ns_span_attn_workspace_bytes(head_dim: int = 64) -> int:
    return int(lib().ns_span_attn_workspace_bytes(head_dim))


def alloc_span_workspace(head_dim: int = 64, device=None) -> torch.Tensor:
    """A workspace for ns_prompt_attn and ns_paged_attn_prefill_q8_0 (its contents need no initialisation)."""
    return torch.empty(ns_span_attn_workspace_bytes(head_dim), dtype=torch.uint8, device=device or "cuda")


def ns_prompt_attn(q, k, v, query_start_loc, scale, out, workspace, key_start_loc=None, stream=None):
    """Causal attention of packed prompts: q [T, Hq, D] over k and v [T', Hkv, D] (rows any stride
    apart); sequence s owns the rows query_start_loc[s]..[s+1] (int32 [S+1]) of q, and of k and v
    unless key_start_loc says otherwise."""
    rows, keys, starts = q.shape, k.shape, query_start_loc.shape
    if len(rows) != 3 or len(keys) != 3 or v.shape != keys or keys[2] != rows[2]:
        raise ValueError("q must be [T, Hq, D], k and v [T', Hkv, D]")
    T, hq, d = rows
    Tk, hkv, _ = keys
    if out.shape != rows:
        raise ValueError("out must have q's shape")
    if len(starts) != 1 or starts[0] < 1:
        raise ValueError("query_start_loc must be [num_seqs + 1]")
    S = starts[0] - 1
    if key_start_loc is None:
        if Tk != T:
            raise ValueError("k and v must have q's rows when key_start_loc is not given")
    elif key_start_loc.shape != starts:
        raise ValueError("key_start_loc must be [num_seqs + 1]")
    dtype = q.dtype
    dt = _dtype_code(q)
    (qp, qs), (kp, ks), (vp, vs) = _rows(q, "q", dtype, rows), _rows(k, "k", dtype, keys), _rows(v, "v", dtype, keys)
    st = _invoke("ns_prompt_attn", qp, kp, vp, _dev(query_start_loc, "query_start_loc", torch.int32),
                 None if key_start_loc is None else _dev(key_start_loc, "key_start_loc", torch.int32),
                 S, T, Tk, hq, hkv, d, qs, ks, vs, float(scale), _dev(out, "out", dtype), _stream(stream), dt,
                 _dev(workspace, "workspace", torch.uint8), workspace.numel())
    _check(st, "ns_prompt_attn")


def ns_paged_attn_prefill_q8_0(q, query_start_loc, k_codes, k_scales, v_codes, v_scales, block_tables,
                               context_lens, scale, out, workspace, stream=None):
    """Attention of the query spans ``query_start_loc`` over a q8_0 pool (block size 16); the workspace
    is alloc_span_workspace's."""
    T, hq, d = q.shape
    nb, hkv, bs, d2, kc, ks, vc, vs = _q8_pools(k_codes, k_scales, v_codes, v_scales)
    S = context_lens.shape[0]
    if d2 != d or out.shape != q.shape or query_start_loc.shape != (S + 1,) or block_tables.dim() != 2 \
            or block_tables.shape[0] != S:
        raise ValueError("shape mismatch")
    st = _invoke("ns_paged_attn_prefill_q8_0",
                 _dev(q, "q"), _dev(query_start_loc, "query_start_loc", torch.int32), kc, ks, vc, vs,
                 _dev(block_tables, "block_tables", torch.int32), _dev(context_lens, "context_lens", torch.int32),
                 S, T, hq, hkv, d, bs, float(scale), _dev(out, "out", q.dtype), _stream(stream),
                 block_tables.shape[1], nb, _dtype_code(q), _dev(workspace, "workspace", torch.uint8),
                 workspace.numel())
    _check(st, "ns_paged_attn_prefill_q8_0")


def _gather_shapes(hkv, d, block_tables, start_loc, k_out, v_out):
    """(num_seqs, max_blocks_per_seq, total_tokens, type) of a read-back."""
    out, tables, dtype = k_out.shape, block_tables.shape, k_out.dtype
    if len(out) != 3 or out[1] != hkv or out[2] != d or v_out.shape != out or v_out.dtype is not dtype:
        raise ValueError("k_out and v_out must be [total_tokens, Hkv, D]")
    if len(tables) != 2 or start_loc.shape != (tables[0] + 1,):
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq], start_loc [num_seqs + 1]")
    return tables[0], tables[1], out[0], dtype


def ns_kv_gather(k_pool, v_pool, block_tables, start_loc, k_out, v_out, stream=None):
    """Read the first start_loc[s+1]-start_loc[s] tokens of each sequence from the pools into the
    packed rows k_out/v_out [T, Hkv, D]."""
    pool = k_pool.shape
    nb, hkv, bs, d = pool
    if v_pool.shape != pool:
        raise ValueError("shape mismatch")
    S, width, T, dtype = _gather_shapes(hkv, d, block_tables, start_loc, k_out, v_out)
    st = _invoke("ns_kv_gather", _dev(k_pool, "k_pool", dtype), _dev(v_pool, "v_pool", dtype),
                 _dev(block_tables, "block_tables", torch.int32), _dev(start_loc, "start_loc", torch.int32),
                 S, T, hkv, d, bs, _dev(k_out, "k_out"), _dev(v_out, "v_out"), _stream(stream), width, nb,
                 _dtype_code(k_out))
    _check(st, "ns_kv_gather")


def ns_kv_gather_q8_0(k_codes, k_scales, v_codes, v_scales, block_tables, start_loc, k_out, v_out, stream=None):
    """ns_kv_gather from a q8_0 pool: the dequantised rows, rounded to k_out's type."""
    nb, hkv, bs, d, kc, ks, vc, vs = _q8_pools(k_codes, k_scales, v_codes, v_scales)
    S, width, T, _ = _gather_shapes(hkv, d, block_tables, start_loc, k_out, v_out)
    st = _invoke("ns_kv_gather_q8_0", kc, ks, vc, vs, _dev(block_tables, "block_tables", torch.int32),
                 _dev(start_loc, "start_loc", torch.int32), S, T, hkv, d, bs, _dev(k_out, "k_out"),
                 _dev(v_out, "v_out"), _stream(stream), width, nb, _dtype_code(k_out))
    _check(st, "ns_kv_gather_q8_0")


def _prob_rows(t, name, shape):
    if t.dtype is not torch.float32:
        raise TypeError(f"{name} must be torch.float32, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    n, width = shape
    s0, s1 = t.stride()
    if n and width > 1 and s1 != 1:
        raise ValueError(f"the rows of {name} must be dense")
    return t.data_ptr(), (s0 if n > 1 else width)


def ns_verify_drafts(target_probs, draft_probs, draft_tokens, draft_start_loc, accept_uniforms, sample_uniforms,
                     out_tokens, num_accepted, stream=None):
    """Verify the drafted tokens of each sequence against the target's probabilities.

    target_probs float32 [T + S, V] (a sequence of n drafts has n + 1 rows), draft_probs [T, V] or
    None (certain drafts), draft_tokens int32 [T], draft_start_loc int32 [S + 1], uniforms in [0, 1).
    Writes out_tokens int32 [T + S] (accepted drafts, the drawn token, then -1) and num_accepted [S].
    """
    target, drafts, accepted = target_probs.shape, draft_tokens.shape, num_accepted.shape
    if len(drafts) != 1 or len(accepted) != 1:
        raise ValueError("draft_tokens must be [num_drafts], num_accepted [num_seqs]")
    T, S = drafts[0], accepted[0]
    if len(target) != 2 or target[0] != T + S or out_tokens.shape != (T + S,):
        raise ValueError("target_probs must be [num_drafts + num_seqs, V], out_tokens [num_drafts + num_seqs]")
    V = target[1]
    if draft_probs is not None and draft_probs.shape != (T, V):
        raise ValueError("draft_probs must be [num_drafts, V]")
    if draft_start_loc.shape != (S + 1,) or accept_uniforms.shape != (T,) or sample_uniforms.shape != (S,):
        raise ValueError("draft_start_loc must be [S + 1], accept_uniforms [num_drafts], sample_uniforms [S]")
    p, ps = _prob_rows(target_probs, "target_probs", target)
    q, qs = (None, 0) if draft_probs is None else _prob_rows(draft_probs, "draft_probs", (T, V))
    st = _invoke("ns_verify_drafts", p, q, _dev(draft_tokens, "draft_tokens", torch.int32),
                 _dev(draft_start_loc, "draft_start_loc", torch.int32),
                 _dev(accept_uniforms, "accept_uniforms", torch.float32),
                 _dev(sample_uniforms, "sample_uniforms", torch.float32), S, T, V, ps, qs,
                 _dev(out_tokens, "out_tokens", torch.int32), _dev(num_accepted, "num_accepted", torch.int32),
                 _stream(stream))
    _check(st, "ns_verify_drafts")


def ns_read_decode_plan(workspace, stream=None) -> dict:
    plan = DecodePlan()
    _check(lib().ns_read_decode_plan(_dev(workspace, "workspace", torch.uint8), ctypes.byref(plan),
                                     _stream(stream)), "ns_read_decode_plan")
    return {f: getattr(plan, f) for f, _ in DecodePlan._fields_ if f != "reserved"}


def ns_get_device_status(clear: bool = True, stream=None) -> int:
    bits = ctypes.c_uint32(0)
    _check(lib().ns_get_device_status(_stream(stream), ctypes.byref(bits), int(bool(clear))),
           "ns_get_device_status")
    return int(bits.value)


def raise_on_device_status(stream=None):
    """Raise NsError(NS_ERR_DEVICE) if a kernel raised a device status bit (and clear it)."""
    bits = ns_get_device_status(clear=True, stream=stream)
    if bits:
        names = [n for b, n in DEV_BITS.items() if bits & b]
        raise RuntimeError(f"device status 0x{bits:x}: {', '.join(names)}")
