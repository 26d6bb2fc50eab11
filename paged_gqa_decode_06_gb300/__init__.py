"""Paged grouped-query decode attention for GB300 (sm_103a).

Thin binding over the C ABI in ``include/decode_attn.h`` (the shared library
``_build/libpaged_gqa_decode.so``, built by ``build.build()``).  This module
only marshals arguments: torch tensors become raw device pointers, the
current CUDA stream becomes the ``stream`` argument, and the workspace is a
torch allocation cached per device and stream.  Every step of the computation runs in
the library's CUDA kernels; there is no other code path, and calling any
entry point without the built library raises.

Entry points (same names as the C ABI):
  decode_attn, decode_attn_split, decode_attn_combine, decode_attn_host,
  decode_attn_workspace_size, decode_attn_make_plan, decode_attn_strerror;
  decode_attn_chunk (attention of a ragged batch of new tokens);
  decode_kv_append_chunk, decode_kv_read (a chunk's rows into a 16- or 8-bit
  paged cache and back), decode_attn_quant (the decode step over an 8-bit one)
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional

try:
    import torch
except ImportError:  # the C ABI and the planners need no torch
    torch = None

__all__ = [
    "DecodeAttnParams", "DecodeAttnPlan", "DecodeAttnError", "load_library", "library_path",
    "make_params", "decode_attn", "decode_attn_split", "decode_attn_combine",
    "decode_attn_host", "decode_attn_workspace_size", "decode_attn_make_plan",
    "decode_attn_strerror", "VARIANT_AUTO", "VARIANT_SIMT", "VARIANT_MMA",
    "DEV_BAD_LEN", "DEV_BAD_PAGE", "DEV_OVER_HINT", "DEV_TIMEOUT", "DEV_CHECK",
    "decode_attn_static_scratch", "decode_attn_workspace_clear", "DEV_WORKSPACE",
    "decode_kv_append", "decode_attn_append", "DTYPE_FP16", "DTYPE_BF16",
    "SCHEDULE_AUTO", "SCHEDULE_GRID", "SCHEDULE_CLUSTER",
    "DecodeAttnChunkPlan", "decode_attn_chunk", "decode_attn_chunk_make_plan",
    "decode_attn_chunk_workspace_size", "KV_16BIT", "KV_E4M3", "decode_kv_append_chunk",
    "decode_kv_read", "decode_attn_quant", "decode_attn_quant_make_plan",
    "decode_attn_quant_workspace_size",
]

VARIANT_AUTO, VARIANT_SIMT, VARIANT_MMA = 0, 1, 2
SCHEDULE_AUTO, SCHEDULE_GRID, SCHEDULE_CLUSTER = 0, 1, 2
DTYPE_FP16, DTYPE_BF16 = 0, 1
KV_16BIT, KV_E4M3 = 0, 1
DEV_BAD_LEN, DEV_BAD_PAGE, DEV_OVER_HINT, DEV_TIMEOUT, DEV_WORKSPACE = 1, 2, 4, 8, 16
DEV_CHECK = 32  # the checked build only: an index outside its buffer

_HERE = os.path.dirname(os.path.abspath(__file__))


def library_path() -> str:
    """The library this process loads: the checked build (bounds-checked
    kernels) when DECODE_ATTN_CHECKED=1, else the release build."""
    if os.environ.get("DECODE_ATTN_CHECKED") == "1":
        return os.path.join(_HERE, "_build_checked", "libpaged_gqa_decode_checked.so")
    return os.path.join(_HERE, "_build", "libpaged_gqa_decode.so")


class DecodeAttnParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_q_heads", "num_kv_heads", "head_dim", "page_size",
        "max_pages_per_seq", "num_pages", "max_seq_len")] + [
        ("scale", ctypes.c_float), ("window", ctypes.c_int32), ("variant", ctypes.c_int32),
        ("split_min", ctypes.c_int32), ("force_chunk", ctypes.c_int32),
        ("num_queries", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("schedule", ctypes.c_int32)]


class DecodeAttnPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "split", "variant", "group_pad", "tile_tokens", "chunk_tokens", "max_shards",
        "grid_x", "grid_y", "grid_z", "ctas_per_sm", "head_fastest", "ring_stages",
        "cluster", "balanced")] + [
        ("workspace_bytes", ctypes.c_size_t)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class DecodeAttnChunkPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "tile_tokens", "item_tokens", "slots", "max_shards", "shard_keys", "grid")] + [
        ("workspace_bytes", ctypes.c_size_t)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class DecodeAttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {decode_attn_strerror(code)} (status {code})")
        self.code = code


_lib = None
_lock = threading.Lock()


def load_library():
    """The CUDA library, loaded once.  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"CUDA library not built ({path} missing); run "
                    "paged_gqa_decode_06_gb300.build.build()")
            lib = ctypes.CDLL(path)
            P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
            PP = ctypes.POINTER(DecodeAttnParams)
            lib.decode_attn_make_plan.argtypes = [PP, i32, ctypes.POINTER(DecodeAttnPlan)]
            lib.decode_attn_make_plan.restype = ctypes.c_int
            lib.decode_attn_workspace_size.argtypes = [PP, ctypes.c_int]
            lib.decode_attn_workspace_size.restype = sz
            for name in ("decode_attn", "decode_attn_split"):
                f = getattr(lib, name)
                f.argtypes = [PP, P, P, P, P, P, P, P, sz, P, P]
                f.restype = ctypes.c_int
            lib.decode_attn_combine.argtypes = [PP, P, P, P, sz, P, P]
            lib.decode_attn_combine.restype = ctypes.c_int
            lib.decode_attn_host.argtypes = [PP] + [P] * 12 + [sz, P, sz, P, P]
            lib.decode_attn_host.restype = ctypes.c_int
            lib.decode_kv_append.argtypes = [PP, P, P, P, P, P, P, P, P]
            lib.decode_kv_append.restype = ctypes.c_int
            lib.decode_attn_append.argtypes = [PP, P, P, P, P, P, P, P, P, P, sz, P, P]
            lib.decode_attn_append.restype = ctypes.c_int
            lib.decode_attn_workspace_clear.argtypes = [PP, P, sz, P]
            lib.decode_attn_workspace_clear.restype = ctypes.c_int
            lib.decode_attn_chunk_make_plan.argtypes = [PP, i32, i32,
                                                        ctypes.POINTER(DecodeAttnChunkPlan)]
            lib.decode_attn_chunk_make_plan.restype = ctypes.c_int
            lib.decode_attn_chunk_workspace_size.argtypes = [PP, i32, ctypes.c_int]
            lib.decode_attn_chunk_workspace_size.restype = sz
            lib.decode_attn_chunk.argtypes = [PP, i32, P, P, P, P, P, P, P, P, sz, P, P]
            lib.decode_attn_chunk.restype = ctypes.c_int
            lib.decode_kv_append_chunk.argtypes = [PP, i32, i32] + [P] * 11
            lib.decode_kv_append_chunk.restype = ctypes.c_int
            lib.decode_kv_read.argtypes = [PP, i32, i32] + [P] * 11
            lib.decode_kv_read.restype = ctypes.c_int
            lib.decode_attn_quant_make_plan.argtypes = [PP, i32, i32,
                                                        ctypes.POINTER(DecodeAttnPlan)]
            lib.decode_attn_quant_make_plan.restype = ctypes.c_int
            lib.decode_attn_quant_workspace_size.argtypes = [PP, i32, ctypes.c_int]
            lib.decode_attn_quant_workspace_size.restype = sz
            lib.decode_attn_quant.argtypes = [PP, i32, P, P, P, P, P, P, P, P, P, sz, P, P]
            lib.decode_attn_quant.restype = ctypes.c_int
            lib.decode_attn_strerror.argtypes = [ctypes.c_int]
            lib.decode_attn_strerror.restype = ctypes.c_char_p
            _lib = lib
    return _lib


def _on_device_of(name: str, index: int):
    """Runs the wrapped call with the CUDA device of its tensor argument
    `name` (positional `index`) current: the library launches on the current
    device, and the default stream is that device's current stream, so
    tensors on another GPU than the current one still get their own device."""
    def deco(fn):
        @functools.wraps(fn)
        def wrapper(*args, **kwargs):
            import torch
            t = kwargs.get(name, args[index] if len(args) > index else None)
            if isinstance(t, torch.Tensor) and t.is_cuda and \
                    t.device.index not in (None, torch.cuda.current_device()):
                with torch.cuda.device(t.device):
                    return fn(*args, **kwargs)
            return fn(*args, **kwargs)
        return wrapper
    return deco


def decode_attn_strerror(code: int) -> str:
    return load_library().decode_attn_strerror(int(code)).decode()


def make_params(q, k_pages, page_table, scale: float, window: int = 0,
                max_seq_len: Optional[int] = None, variant: int = VARIANT_AUTO,
                split_min: int = 0, force_chunk: int = 0,
                schedule: int = SCHEDULE_AUTO) -> DecodeAttnParams:
    """Parameters from tensor shapes: q [B,Hq,D] (or [B,T,Hq,D] for T query
    positions per sequence), k_pages [P,PS,Hkv,D], page_table [B,maxPages].
    ``max_seq_len`` is a host-side bound on seq_lens (it sizes the grid;
    None = the page table's capacity).  ``schedule``: SCHEDULE_AUTO (the
    planner's grid or cluster plan), SCHEDULE_GRID or SCHEDULE_CLUSTER (a
    schedule the shape cannot take raises DecodeAttnError at planning)."""
    if len(q.shape) == 4:
        B, T, Hq, D = q.shape
    else:
        (B, Hq, D), T = q.shape, 1
    P, PS, Hkv, D2 = k_pages.shape
    if D2 != D:
        raise ValueError("q and k_pages head_dim differ")
    return DecodeAttnParams(
        batch=B, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=PS,
        max_pages_per_seq=page_table.shape[1], num_pages=P,
        max_seq_len=int(max_seq_len) if max_seq_len else 0, scale=float(scale),
        window=int(window), variant=int(variant), split_min=int(split_min),
        force_chunk=int(force_chunk), num_queries=int(T), dtype=_dtype_code(q),
        schedule=int(schedule))


def _dtype_code(t) -> int:
    """DTYPE_BF16 for torch.bfloat16 tensors, else DTYPE_FP16."""
    return DTYPE_BF16 if str(getattr(t, "dtype", "")) == "torch.bfloat16" else DTYPE_FP16


def _elem_dtype(t):
    import torch
    if t.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"expected float16 or bfloat16 tensors, got {t.dtype}")
    return t.dtype


def decode_attn_make_plan(params: DecodeAttnParams, num_sms: int) -> DecodeAttnPlan:
    plan = DecodeAttnPlan()
    st = load_library().decode_attn_make_plan(ctypes.byref(params), int(num_sms),
                                              ctypes.byref(plan))
    if st:
        raise DecodeAttnError(st, "decode_attn_make_plan")
    return plan


def decode_attn_workspace_size(params: DecodeAttnParams, device: int) -> int:
    return int(load_library().decode_attn_workspace_size(ctypes.byref(params), int(device)))


@_on_device_of("workspace", 1)
def decode_attn_workspace_clear(params: DecodeAttnParams, workspace, stream=None) -> None:
    """Zeroes the workspace's shard tickets (needed once for a workspace that
    was not allocated zero-filled, or after a DEV_TIMEOUT / DEV_WORKSPACE)."""
    nbytes = workspace.numel() * workspace.element_size()
    st = load_library().decode_attn_workspace_clear(ctypes.byref(params), _ptr(workspace),
                                                    nbytes, _stream_handle(stream))
    if st:
        raise DecodeAttnError(st, "decode_attn_workspace_clear")


# ------------------------------------------------------------ torch glue

_ws_cache: dict = {}


def _workspace(device, nbytes: int, stream=None):
    """The cached workspace of (device, stream): calls on different streams
    may run at the same time, so each stream has its own tickets and
    partials.  A buffer is allocated zero-filled on the stream it serves, so
    the fill is ordered before that stream's kernels (and a replaced buffer
    is only reused by later work of the same stream)."""
    import torch
    if nbytes == 0:
        return None
    index = device.index if device.index is not None else torch.cuda.current_device()
    s = stream if stream is not None else torch.cuda.current_stream(index)
    key = (index, s.cuda_stream)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        # zero-filled: its shard tickets must start at zero (the kernels leave
        # them zero after every completed call)
        with torch.cuda.stream(s):
            buf = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check(t, dtype, name, device=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _stream_handle(stream) -> int:
    """The raw handle of `stream`, by default the current device's current
    stream; a stream of another device than the current one is refused."""
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if stream.device.index != torch.cuda.current_device():
        raise ValueError(f"stream is on {stream.device}, the tensors on "
                         f"cuda:{torch.cuda.current_device()}")
    return stream.cuda_stream


def _new_like(t, stream=None):
    """A new output like ``t`` that a call on ``stream`` fills: allocated on
    that stream, since memory that the current stream's allocator hands out
    may still be in use by that stream's earlier work."""
    if stream is None:
        return torch.empty_like(t)
    with torch.cuda.stream(stream):
        return torch.empty_like(t)


def _prepare(q, k_pages, v_pages, page_table, seq_lens, out, scale, window, max_seq_len,
             variant, split_min, force_chunk, workspace, schedule=SCHEDULE_AUTO, stream=None):
    import torch
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("decode_attn runs on CUDA tensors (use decode_attn_host for host "
                         "buffers)")
    et = _elem_dtype(q)
    _check(q, et, "q", dev)
    _check(k_pages, et, "k_pages", dev)
    _check(v_pages, et, "v_pages", dev)
    _check(page_table, torch.int32, "page_table", dev)
    _check(seq_lens, torch.int32, "seq_lens", dev)
    if v_pages.shape != k_pages.shape:
        raise ValueError("k_pages and v_pages shapes differ")
    p = make_params(q, k_pages, page_table, scale, window, max_seq_len, variant, split_min,
                    force_chunk, schedule)
    if out is None:
        out = _new_like(q, stream)
    _check(out, et, "out", dev)
    need = decode_attn_workspace_size(p, dev.index if dev.index is not None else
                                      torch.cuda.current_device())
    if workspace is None:
        workspace = _workspace(dev, need, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return p, out, workspace, ws_bytes


@_on_device_of("q", 0)
def decode_attn(q, k_pages, v_pages, page_table, seq_lens, scale: float, window: int = 0,
                out=None, max_seq_len: Optional[int] = None, workspace=None, err_flag=None,
                variant: int = VARIANT_AUTO, split_min: int = 0, force_chunk: int = 0,
                stream=None, schedule: int = SCHEDULE_AUTO):
    """One decode step of paged GQA attention; returns ``out`` [B,Hq,D] fp16.

    q [B,Hq,D] fp16, k_pages/v_pages [P,PS,Hkv,D] fp16, page_table [B,maxPages]
    int32, seq_lens [B] int32, all on one CUDA device.  ``window`` > 0 attends
    the last min(L, window) positions.  ``err_flag``: optional int32 device
    tensor of one element that receives DEV_* bits.  Enqueued on ``stream``
    (default: torch's current stream), in whose memory a new ``out`` lies; does
    not synchronise.  ``workspace``: by default a zero-filled buffer cached per
    (device, stream); pass one to keep its fill out of a captured graph."""
    p, out, ws, ws_bytes = _prepare(q, k_pages, v_pages, page_table, seq_lens, out, scale,
                                    window, max_seq_len, variant, split_min, force_chunk,
                                    workspace, schedule, stream)
    st = load_library().decode_attn(ctypes.byref(p), _ptr(q), _ptr(k_pages), _ptr(v_pages),
                                    _ptr(page_table), _ptr(seq_lens), _ptr(out), _ptr(ws),
                                    ws_bytes, _ptr(err_flag), _stream_handle(stream))
    if st:
        raise DecodeAttnError(st, "decode_attn")
    return out


@_on_device_of("k_pages", 3)
def decode_kv_append(k_new, v_new, positions, k_pages, v_pages, page_table, err_flag=None,
                     stream=None):
    """Writes the step's new rows k_new/v_new [B,Hkv,D] at positions[b]
    (int32, -1 = none) into the paged pools, bit for bit."""
    import torch
    dev = k_pages.device
    et = _elem_dtype(k_pages)
    _check(k_new, et, "k_new", dev)
    _check(v_new, et, "v_new", dev)
    _check(positions, torch.int32, "positions", dev)
    _check(k_pages, et, "k_pages", dev)
    _check(v_pages, et, "v_pages", dev)
    _check(page_table, torch.int32, "page_table", dev)
    P, PS, Hkv, D = k_pages.shape
    if tuple(k_new.shape) != (page_table.shape[0], Hkv, D) or v_new.shape != k_new.shape:
        raise ValueError("k_new / v_new must be [B, Hkv, D]")
    p = DecodeAttnParams(batch=page_table.shape[0], num_q_heads=Hkv, num_kv_heads=Hkv,
                         head_dim=D, page_size=PS, max_pages_per_seq=page_table.shape[1],
                         num_pages=P, max_seq_len=0, scale=1.0, window=0, variant=0,
                         split_min=0, force_chunk=0, num_queries=1, dtype=_dtype_code(k_pages),
                         schedule=0)
    st = load_library().decode_kv_append(ctypes.byref(p), _ptr(k_new), _ptr(v_new),
                                         _ptr(positions), _ptr(k_pages), _ptr(v_pages),
                                         _ptr(page_table), _ptr(err_flag),
                                         _stream_handle(stream))
    if st:
        raise DecodeAttnError(st, "decode_kv_append")


@_on_device_of("q", 0)
def decode_attn_append(q, k_new, v_new, k_pages, v_pages, page_table, seq_lens, scale: float,
                       window: int = 0, out=None, max_seq_len: Optional[int] = None,
                       workspace=None, err_flag=None, variant: int = VARIANT_AUTO,
                       split_min: int = 0, force_chunk: int = 0, stream=None,
                       schedule: int = SCHEDULE_AUTO):
    """Append + attention in one launch: writes k_new/v_new [B,Hkv,D] (or
    [B,T,Hkv,D] with q [B,T,Hq,D]) at the last T positions of each sequence
    (seq_lens counts them), then attends as decode_attn."""
    import torch
    p, out, ws, ws_bytes = _prepare(q, k_pages, v_pages, page_table, seq_lens, out, scale,
                                    window, max_seq_len, variant, split_min, force_chunk,
                                    workspace, schedule, stream)
    _check(k_new, q.dtype, "k_new", q.device)
    _check(v_new, q.dtype, "v_new", q.device)
    st = load_library().decode_attn_append(ctypes.byref(p), _ptr(q), _ptr(k_new), _ptr(v_new),
                                           _ptr(k_pages), _ptr(v_pages), _ptr(page_table),
                                           _ptr(seq_lens), _ptr(out), _ptr(ws), ws_bytes,
                                           _ptr(err_flag), _stream_handle(stream))
    if st:
        raise DecodeAttnError(st, "decode_attn_append")
    return out


@_on_device_of("q", 0)
def decode_attn_split(q, k_pages, v_pages, page_table, seq_lens, scale: float, window: int = 0,
                      out=None, max_seq_len=None, workspace=None, err_flag=None,
                      variant: int = VARIANT_AUTO, split_min: int = 0, force_chunk: int = 0,
                      stream=None, schedule: int = SCHEDULE_AUTO):
    """The shard kernel alone (writes ``out`` directly for a single-pass plan,
    partials into ``workspace`` otherwise).  Returns (out, workspace)."""
    p, out, ws, ws_bytes = _prepare(q, k_pages, v_pages, page_table, seq_lens, out, scale,
                                    window, max_seq_len, variant, split_min, force_chunk,
                                    workspace, schedule, stream)
    st = load_library().decode_attn_split(ctypes.byref(p), _ptr(q), _ptr(k_pages),
                                          _ptr(v_pages), _ptr(page_table), _ptr(seq_lens),
                                          _ptr(out), _ptr(ws), ws_bytes, _ptr(err_flag),
                                          _stream_handle(stream))
    if st:
        raise DecodeAttnError(st, "decode_attn_split")
    return out, ws


@_on_device_of("out", 2)
def decode_attn_combine(params: DecodeAttnParams, seq_lens, out, workspace, err_flag=None,
                        stream=None):
    """The ordered combine alone, for ``params`` as used by decode_attn_split."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load_library().decode_attn_combine(ctypes.byref(params), _ptr(seq_lens), _ptr(out),
                                            _ptr(workspace), ws_bytes, _ptr(err_flag),
                                            _stream_handle(stream))
    if st:
        raise DecodeAttnError(st, "decode_attn_combine")
    return out


@_on_device_of("d_q", 7)
def decode_attn_host(params: DecodeAttnParams, q_host, k_host, v_host, table_host, lens_host,
                     out_host, d_q, d_k, d_v, d_table, d_lens, d_out, workspace,
                     kv_bytes_to_copy: int = 0, err_flag=None, stream=None):
    """End-to-end step from host buffers (pinned CPU tensors): copies in,
    decode_attn, copies ``out`` back; enqueued on ``stream``, not awaited."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load_library().decode_attn_host(
        ctypes.byref(params), _ptr(q_host), _ptr(k_host), _ptr(v_host), _ptr(table_host),
        _ptr(lens_host), _ptr(out_host), _ptr(d_q), _ptr(d_k), _ptr(d_v), _ptr(d_table),
        _ptr(d_lens), _ptr(d_out), int(kv_bytes_to_copy), _ptr(workspace), ws_bytes,
        _ptr(err_flag), _stream_handle(stream))
    if st:
        raise DecodeAttnError(st, "decode_attn_host")
    return out_host


# ------------------------------------------- no-allocation variant

def _static_scratch_fn():
    f = load_library().decode_attn_static_scratch
    if f.argtypes is None:
        P = ctypes.c_void_p
        f.argtypes = [ctypes.POINTER(DecodeAttnParams), P, P, P, P, P, P, P, P]
        f.restype = ctypes.c_int
    return f


@_on_device_of("q", 0)
def decode_attn_static_scratch(q, k_pages, v_pages, page_table, seq_lens, scale: float,
                               window: int = 0, out=None, max_seq_len: Optional[int] = None,
                               err_flag=None, variant: int = VARIANT_AUTO, split_min: int = 0,
                               force_chunk: int = 0, stream=None,
                               schedule: int = SCHEDULE_AUTO):
    """decode_attn for callers that cannot allocate device memory: the shard
    partials use the library's fixed 8 MiB device array instead of a
    workspace (shared by all calls on a device; overlapping calls race).
    Only ``out`` is created here when not given; pass it to allocate nothing."""
    import torch
    dev = q.device
    et = _elem_dtype(q)
    for t, dt, n in ((q, et, "q"), (k_pages, et, "k_pages"), (v_pages, et, "v_pages"),
                     (page_table, torch.int32, "page_table"), (seq_lens, torch.int32, "seq_lens")):
        _check(t, dt, n, dev)
    if out is None:
        out = _new_like(q, stream)
    _check(out, et, "out", dev)
    p = make_params(q, k_pages, page_table, scale, window, max_seq_len, variant, split_min,
                    force_chunk, schedule)
    st = _static_scratch_fn()(ctypes.byref(p), _ptr(q), _ptr(k_pages), _ptr(v_pages),
                              _ptr(page_table), _ptr(seq_lens), _ptr(out), _ptr(err_flag),
                              _stream_handle(stream))
    if st:
        raise DecodeAttnError(st, "decode_attn_static_scratch")
    return out


# ------------------------------------------------ new tokens by the chunk
#
# A small call is bound by what the host does before its launch, so these
# functions look at each tensor once and leave the wording of an error to the
# slower checks.

def _need(t, dtype, name, index):
    """A contiguous tensor of this type on CUDA device `index`."""
    if not (type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == index and
            t.is_contiguous()):
        _check(t, dtype, name, torch.device("cuda", index) if index >= 0 else None)


def _cuda_index(t, name: str, call: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{call} runs on CUDA tensors")
    return t.get_device()


def _raw_stream(stream, index: int) -> int:
    """_stream_handle for tensors on the current device `index`."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return _stream_handle(stream)


def _scratch(index: int, nbytes: int, zero: bool, stream):
    """A workspace for one call: cached per (device, stream) like
    decode_attn's, but a call under stream capture gets one of its own, so
    that two captured graphs never share one."""
    if nbytes == 0:
        return None
    if stream is not None and stream != torch.cuda.current_stream(index):
        with torch.cuda.stream(stream):
            return _scratch(index, nbytes, zero, None)
    capturing = torch.cuda.is_current_stream_capturing()
    key = (index, _raw_stream(None, index), zero)
    buf = None if capturing else _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        make = torch.zeros if zero else torch.empty
        buf = make(max(nbytes, 1 << 20), dtype=torch.uint8, device=torch.device("cuda", index))
        if not capturing:
            _ws_cache[key] = buf
    return buf


def _check_offsets(t, batch: int, name: str, index: int):
    _need(t, torch.int32, name, index)
    if t.shape != (batch + 1,):
        raise ValueError(f"{name} must be [B + 1] = [{batch + 1}], got {list(t.shape)}")


def _check_table(page_table, seq_lens, index: int) -> int:
    """The batch, after checking the table (and the lengths, if any)."""
    _need(page_table, torch.int32, "page_table", index)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    batch = page_table.shape[0]
    if seq_lens is not None:
        _need(seq_lens, torch.int32, "seq_lens", index)
        if seq_lens.shape != (batch,):
            raise ValueError(f"seq_lens must be [B] = [{batch}]")
    return batch


def _err_ptr(err_flag, index: int) -> Optional[int]:
    if err_flag is None:
        return None
    _need(err_flag, torch.int32, "err_flag", index)
    return err_flag.data_ptr()


def _ws_args(workspace, index: int):
    if workspace is None:
        return None, 0
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on cuda:{index}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _kv_pools(k_pages, v_pages, k_scales, v_scales, index: int) -> int:
    """The cell format of a pair of pools, after checking them (and the
    scales an 8-bit pair needs)."""
    if not isinstance(k_pages, torch.Tensor):
        raise TypeError("k_pages must be a torch.Tensor")
    dt, shape = k_pages.dtype, k_pages.shape
    quant = dt is torch.float8_e4m3fn
    if not quant:
        _elem_dtype(k_pages)
    _need(k_pages, dt, "k_pages", index)
    _need(v_pages, dt, "v_pages", index)
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must be [P, PS, Hkv, D], both of one shape")
    if not quant:
        if k_scales is not None or v_scales is not None:
            raise ValueError("k_scales and v_scales go with float8_e4m3fn pools only")
        return KV_16BIT
    if k_scales is None or v_scales is None:
        raise ValueError("float8_e4m3fn pools need k_scales and v_scales")
    _need(k_scales, torch.float32, "k_scales", index)
    _need(v_scales, torch.float32, "v_scales", index)
    want = (shape[0], shape[2], shape[1])
    if k_scales.shape != want or v_scales.shape != want:
        raise ValueError(f"k_scales and v_scales must be [P, Hkv, PS] = {list(want)}")
    return KV_E4M3


def _params(B, Hq, pool_shape, max_pages, max_seq_len, scale, window, dtype, split_min=0,
            force_chunk=0, T=1, schedule=0) -> DecodeAttnParams:
    P, PS, Hkv, D = pool_shape
    return DecodeAttnParams(B, Hq, Hkv, D, PS, max_pages, P, max_seq_len or 0, scale, window, 0,
                            split_min, force_chunk, T,
                            DTYPE_BF16 if dtype is torch.bfloat16 else DTYPE_FP16, schedule)


def decode_attn_chunk_make_plan(params: DecodeAttnParams, total_queries: int,
                                num_sms: int) -> DecodeAttnChunkPlan:
    plan = DecodeAttnChunkPlan()
    st = load_library().decode_attn_chunk_make_plan(ctypes.byref(params), int(total_queries),
                                                    int(num_sms), ctypes.byref(plan))
    if st:
        raise DecodeAttnError(st, "decode_attn_chunk_make_plan")
    return plan


def decode_attn_chunk_workspace_size(params: DecodeAttnParams, total_queries: int,
                                     device: int) -> int:
    return int(load_library().decode_attn_chunk_workspace_size(
        ctypes.byref(params), int(total_queries), int(device)))


def decode_attn_chunk(q, k_pages, v_pages, page_table, query_offsets, seq_lens, scale: float,
                      window: int = 0, out=None, max_seq_len: Optional[int] = None,
                      workspace=None, err_flag=None, force_chunk: int = 0, stream=None):
    """Attention of a ragged batch of new tokens over the paged cache.

    q [total, Hq, D] fp16 or bf16: sequence b owns the rows query_offsets[b]
    to query_offsets[b + 1] (int32 [B + 1]) and they sit at its last
    positions; seq_lens [B] counts them, and their K/V rows are in the cache
    already.  Token at position p attends the positions up to p, the last
    ``window`` of them with a window.  Returns ``out`` like q; rows that no
    sequence owns keep what they held (a new ``out`` is not initialised).
    ``max_seq_len`` (a host-side bound) only steers the plan."""
    index = _cuda_index(q, "q", "decode_attn_chunk")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return decode_attn_chunk(q, k_pages, v_pages, page_table, query_offsets, seq_lens,
                                     scale, window, out, max_seq_len, workspace, err_flag,
                                     force_chunk, stream)
    et = _elem_dtype(q)
    _need(q, et, "q", index)
    if q.dim() != 3:
        raise ValueError("q must be [total, Hq, D]")
    _need(k_pages, et, "k_pages", index)
    _need(v_pages, et, "v_pages", index)
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("k_pages and v_pages must be [P, PS, Hkv, D], both of one shape")
    if seq_lens is None:
        raise TypeError("seq_lens must be a torch.Tensor")
    B = _check_table(page_table, seq_lens, index)
    _check_offsets(query_offsets, B, "query_offsets", index)
    total, Hq, D = q.shape
    if k_pages.shape[3] != D:
        raise ValueError("q and k_pages head_dim differ")
    if out is None:
        out = _new_like(q, stream)
    else:
        _need(out, et, "out", index)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    p = _params(B, Hq, k_pages.shape, page_table.shape[1], max_seq_len, scale, window, et, 0,
                force_chunk)
    lib, ref = load_library(), ctypes.byref(p)
    if workspace is None:
        workspace = _scratch(index, lib.decode_attn_chunk_workspace_size(ref, total, index),
                             False, stream)
    st = lib.decode_attn_chunk(ref, total, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                               page_table.data_ptr(), query_offsets.data_ptr(),
                               seq_lens.data_ptr(), out.data_ptr(), *_ws_args(workspace, index),
                               _err_ptr(err_flag, index), _raw_stream(stream, index))
    if st:
        raise DecodeAttnError(st, "decode_attn_chunk")
    return out


def decode_kv_append_chunk(k_new, v_new, row_offsets, seq_lens, k_pages, v_pages, page_table,
                           k_scales=None, v_scales=None, err_flag=None, stream=None):
    """Writes a ragged batch's new rows k_new/v_new [total, Hkv, D] (fp16 or
    bf16) into the pools: sequence b owns the rows row_offsets[b] to
    row_offsets[b + 1] and they go to its last positions (seq_lens counts
    them).  16-bit pools get the rows bit for bit; float8_e4m3fn pools get
    codes, and k_scales/v_scales [P, Hkv, PS] float32 a power of two per row
    and head."""
    index = _cuda_index(k_pages, "k_pages", "decode_kv_append_chunk")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return decode_kv_append_chunk(k_new, v_new, row_offsets, seq_lens, k_pages, v_pages,
                                          page_table, k_scales, v_scales, err_flag, stream)
    fmt = _kv_pools(k_pages, v_pages, k_scales, v_scales, index)
    et = _elem_dtype(k_new) if fmt == KV_E4M3 else k_pages.dtype
    _need(k_new, et, "k_new", index)
    _need(v_new, et, "v_new", index)
    if k_new.dim() != 3 or k_new.shape[1:] != k_pages.shape[2:] or v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must be [total, Hkv, D]")
    if seq_lens is None:
        raise TypeError("seq_lens must be a torch.Tensor")
    B = _check_table(page_table, seq_lens, index)
    _check_offsets(row_offsets, B, "row_offsets", index)
    p = _params(B, k_pages.shape[2], k_pages.shape, page_table.shape[1], 0, 1.0, 0, et)
    st = load_library().decode_kv_append_chunk(
        ctypes.byref(p), fmt, k_new.shape[0], k_new.data_ptr(), v_new.data_ptr(),
        row_offsets.data_ptr(), seq_lens.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
        _ptr(k_scales), _ptr(v_scales), page_table.data_ptr(), _err_ptr(err_flag, index),
        _raw_stream(stream, index))
    if st:
        raise DecodeAttnError(st, "decode_kv_append_chunk")


def decode_kv_read(k_pages, v_pages, page_table, row_offsets, total_rows: int, starts=None,
                   k_scales=None, v_scales=None, dtype=None, k_out=None, v_out=None,
                   err_flag=None, stream=None):
    """Reads rows of the paged cache back as contiguous 16-bit rows: output
    row row_offsets[b] + i is position starts[b] + i of sequence b (starts
    None: from 0).  Returns (k, v), [total_rows, Hkv, D] of ``dtype`` (the
    pools' own for 16-bit pools; by default float16 for float8_e4m3fn ones)
    or k_out / v_out as given; rows that no sequence owns keep what they held
    (new outputs are not initialised)."""
    index = _cuda_index(k_pages, "k_pages", "decode_kv_read")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return decode_kv_read(k_pages, v_pages, page_table, row_offsets, total_rows, starts,
                                  k_scales, v_scales, dtype, k_out, v_out, err_flag, stream)
    fmt = _kv_pools(k_pages, v_pages, k_scales, v_scales, index)
    B = _check_table(page_table, None, index)
    _check_offsets(row_offsets, B, "row_offsets", index)
    if starts is not None:
        _need(starts, torch.int32, "starts", index)
        if starts.shape != (B,):
            raise ValueError(f"starts must be [B] = [{B}]")
    if dtype is None:
        given = k_out if k_out is not None else v_out
        dtype = k_pages.dtype if fmt == KV_16BIT else \
            given.dtype if given is not None else torch.float16
    if dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"expected float16 or bfloat16 outputs, got {dtype}")
    if fmt == KV_16BIT and dtype != k_pages.dtype:
        raise TypeError(f"16-bit pools are read back as they are ({k_pages.dtype})")
    shape = (int(total_rows), *k_pages.shape[2:])
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None:
            _need(t, dtype, name, index)
            if t.shape != shape:
                raise ValueError(f"{name} must be [total_rows, Hkv, D] = {list(shape)}")
    if k_out is None and stream is None:
        k_out = torch.empty(shape, dtype=dtype, device=k_pages.device)
    elif k_out is None:  # as _new_like
        with torch.cuda.stream(stream):
            k_out = torch.empty(shape, dtype=dtype, device=k_pages.device)
    if v_out is None:
        v_out = _new_like(k_out, stream)
    p = _params(B, k_pages.shape[2], k_pages.shape, page_table.shape[1], 0, 1.0, 0, dtype)
    st = load_library().decode_kv_read(
        ctypes.byref(p), fmt, shape[0], k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scales),
        _ptr(v_scales), page_table.data_ptr(), row_offsets.data_ptr(), _ptr(starts),
        k_out.data_ptr(), v_out.data_ptr(), _err_ptr(err_flag, index),
        _raw_stream(stream, index))
    if st:
        raise DecodeAttnError(st, "decode_kv_read")
    return k_out, v_out


def decode_attn_quant_make_plan(params: DecodeAttnParams, num_sms: int,
                                kv_format: int = KV_E4M3) -> DecodeAttnPlan:
    plan = DecodeAttnPlan()
    st = load_library().decode_attn_quant_make_plan(ctypes.byref(params), int(kv_format),
                                                    int(num_sms), ctypes.byref(plan))
    if st:
        raise DecodeAttnError(st, "decode_attn_quant_make_plan")
    return plan


def decode_attn_quant_workspace_size(params: DecodeAttnParams, device: int,
                                     kv_format: int = KV_E4M3) -> int:
    return int(load_library().decode_attn_quant_workspace_size(
        ctypes.byref(params), int(kv_format), int(device)))


def decode_attn_quant(q, k_pages, v_pages, k_scales, v_scales, page_table, seq_lens,
                      scale: float, window: int = 0, out=None,
                      max_seq_len: Optional[int] = None, workspace=None, err_flag=None,
                      split_min: int = 0, force_chunk: int = 0, stream=None,
                      schedule: int = SCHEDULE_AUTO):
    """decode_attn over an 8-bit cache: k_pages/v_pages [P, PS, Hkv, D]
    float8_e4m3fn with k_scales/v_scales [P, Hkv, PS] float32 (value = code *
    scale).  q [B, Hq, D] (or [B, T, Hq, D]) fp16 or bf16; returns ``out``
    like q."""
    index = _cuda_index(q, "q", "decode_attn_quant")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return decode_attn_quant(q, k_pages, v_pages, k_scales, v_scales, page_table,
                                     seq_lens, scale, window, out, max_seq_len, workspace,
                                     err_flag, split_min, force_chunk, stream, schedule)
    et = _elem_dtype(q)
    _need(q, et, "q", index)
    if q.dim() == 3:
        (B, Hq, D), T = q.shape, 1
    elif q.dim() == 4:
        B, T, Hq, D = q.shape
    else:
        raise ValueError("q must be [B, Hq, D] or [B, T, Hq, D]")
    if _kv_pools(k_pages, v_pages, k_scales, v_scales, index) != KV_E4M3:
        raise TypeError(f"decode_attn_quant takes float8_e4m3fn pools, got {k_pages.dtype}")
    if k_pages.shape[3] != D:
        raise ValueError("q and k_pages head_dim differ")
    if seq_lens is None:
        raise TypeError("seq_lens must be a torch.Tensor")
    if _check_table(page_table, seq_lens, index) != B:
        raise ValueError("page_table must have a row for each sequence of q")
    if out is None:
        out = _new_like(q, stream)
    else:
        _need(out, et, "out", index)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    p = _params(B, Hq, k_pages.shape, page_table.shape[1], max_seq_len, scale, window, et,
                split_min, force_chunk, T, schedule)
    lib, ref = load_library(), ctypes.byref(p)
    if workspace is None:
        workspace = _scratch(index, lib.decode_attn_quant_workspace_size(ref, KV_E4M3, index),
                             True, stream)
    st = lib.decode_attn_quant(ref, KV_E4M3, q.data_ptr(), k_pages.data_ptr(),
                               v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                               page_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(),
                               *_ws_args(workspace, index), _err_ptr(err_flag, index),
                               _raw_stream(stream, index))
    if st:
        raise DecodeAttnError(st, "decode_attn_quant")
    return out
