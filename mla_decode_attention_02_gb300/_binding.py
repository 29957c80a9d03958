"""Binding over libmla_decode.so: argument marshalling only.

Every step of the computation runs in the library's CUDA kernels; this
module checks tensor shapes, dtypes and devices, allocates the caller-owned
workspace and outputs with PyTorch, and passes raw pointers and the current
CUDA stream through the C ABI declared in include/mla_decode.h, by ctypes.  The
calls of the tree step go first to a C++ module that does the same on torch's
own tensor objects (csrc/host/mla_host.cpp), and come here for what it does not
take.  There is no CPU path: if the library is missing, every call raises.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import threading
import warnings
from dataclasses import dataclass

import numpy as np

NUM_HEADS = 128
D_LATENT = 512
D_ROPE = 64
PAGE_SIZE = 64
DEFAULT_SCALE = 192.0 ** -0.5

MLA_DEV_BAD_PAGE = 0x1
MLA_DEV_BAD_SEQ_LEN = 0x2
MLA_DEV_BAD_PLAN = 0x4
MLA_DEV_TIMEOUT = 0x8

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla_decode.so")

_lock = threading.Lock()
_lib = None


class MLAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_status_string(status)} (status {status})")


class _Problem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("s_q", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("flags", ctypes.c_int32)]


class _Ragged(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("flags", ctypes.c_int32)]


_P = ctypes.POINTER(_Problem)
_R = ctypes.POINTER(_Ragged)
_vp = ctypes.c_void_p
_SIGS = {
    "mla_decode_workspace_size": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_size_t)]),
    "mla_decode_num_units": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int32)]),
    "mla_decode_plan": (ctypes.c_int, [_P, _vp, _vp, ctypes.c_size_t, _vp]),
    "mla_decode": (ctypes.c_int, [_P, _vp, _vp, _vp, ctypes.c_int64, _vp, ctypes.c_float, _vp,
                                  _vp, _vp, ctypes.c_size_t, _vp]),
    "mla_decode_timed": (ctypes.c_int, [_P, _vp, _vp, _vp, ctypes.c_int64, _vp, ctypes.c_float,
                                        _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp]),
    "mla_decode_diag": (ctypes.c_int, [_P, _vp, _vp, _vp, ctypes.c_int64, _vp, ctypes.c_float,
                                       _vp, _vp, _vp, ctypes.c_size_t, _vp, ctypes.c_uint64,
                                       ctypes.c_uint32]),
    "mla_decode_fp8": (ctypes.c_int, [_P, _vp, _vp, _vp, ctypes.c_int64, _vp, ctypes.c_float, _vp,
                                      _vp, _vp, ctypes.c_size_t, _vp, _vp]),
    "mla_decode_noalloc": (ctypes.c_int, [_P, _vp, _vp, _vp, ctypes.c_int64, _vp, _vp,
                                          ctypes.c_float, _vp, _vp, _vp]),
    "mla_decode_check": (ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_int32), _vp]),
    "mla_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "mla_decode_plan_bytes": (ctypes.c_size_t, [_P, ctypes.c_int32]),
    "mla_decode_plan_host": (ctypes.c_int, [_P, _vp, ctypes.c_int32, _vp, ctypes.c_size_t]),
    "mla_prolog": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_float, _vp,
                                  _vp, ctypes.c_int64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "mla_prolog_rope_table": (ctypes.c_int, [ctypes.c_double, _vp, _vp]),
    "mla_epilog_uv": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp]),
    "mla_cache_quantize_fp8": (ctypes.c_int, [_vp, ctypes.c_int64, _vp, _vp]),
    "mla_epilog_oproj": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp]),
    "mla_query": (ctypes.c_int, [ctypes.c_int32, _vp, ctypes.c_int64, ctypes.c_int64, _vp, ctypes.c_int64,
                                 ctypes.c_int64, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "mla_cache_append": (ctypes.c_int, [_R, _vp, ctypes.c_int64, _vp, ctypes.c_int64, _vp, ctypes.c_float, _vp, _vp,
                                        _vp, ctypes.c_int64, _vp, _vp, _vp, _vp, _vp]),
    "mla_tree_workspace_size": (ctypes.c_int, [_R, ctypes.POINTER(ctypes.c_size_t)]),
    "mla_tree_plan": (ctypes.c_int, [_R, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "mla_tree_decode": (ctypes.c_int, [_R, _vp, _vp, _vp, ctypes.c_int64, _vp, ctypes.c_float, _vp, _vp, _vp,
                                       ctypes.c_size_t, _vp]),
    "mla_tree_decode_fp8": (ctypes.c_int, [_R, _vp, _vp, _vp, ctypes.c_int64, _vp, ctypes.c_float, _vp, _vp, _vp,
                                           ctypes.c_size_t, _vp, ctypes.c_size_t, _vp]),
    "mla_tree_scratch_size": (ctypes.c_int, [_R, ctypes.POINTER(ctypes.c_size_t)]),
    "mla_tree_plan_bytes": (ctypes.c_size_t, [_R, ctypes.c_int32]),
    "mla_tree_plan_host": (ctypes.c_int, [_R, _vp, _vp, _vp, ctypes.c_int32, _vp, ctypes.c_size_t]),
    "mla_cache_commit": (ctypes.c_int, [_R, _vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, ctypes.c_int64, _vp,
                                        _vp, _vp, _vp, ctypes.c_int32, _vp, _vp, _vp, _vp]),
}
_SIGS["mla_cache_append_fp8"] = _SIGS["mla_cache_append"]


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libmla_decode.so (built by ``__graft_entry__.build()`` or ``build.py``)."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(
                    f"{p} is missing: build the CUDA library first "
                    "(python -m mla_decode_attention_02_gb300.build); there is no fallback path")
            lib = ctypes.CDLL(p)
            for name, (res, args) in _SIGS.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def _status_string(status: int) -> str:
    try:
        return load_library().mla_status_string(status).decode()
    except Exception:  # pragma: no cover - library not loadable
        return "unknown"


def _check(status: int, what: str) -> None:
    if status != 0:
        raise MLAError(status, what)


MLA_FLAG_POW2_MAX = 0x1


def _problem(batch: int, s_q: int, max_pages: int, flags: int = 0) -> _Problem:
    return _Problem(int(batch), int(s_q), NUM_HEADS, PAGE_SIZE, int(max_pages), int(flags))


def num_units() -> int:
    """Work units (SM groups) the main kernel uses on the current device."""
    u = ctypes.c_int32(0)
    _check(load_library().mla_decode_num_units(ctypes.byref(u)), "mla_decode_num_units")
    return u.value


def workspace_size(batch: int, s_q: int, max_pages: int) -> int:
    n = ctypes.c_size_t(0)
    prob = _problem(batch, s_q, max_pages)
    _check(load_library().mla_decode_workspace_size(ctypes.byref(prob), ctypes.byref(n)),
           "mla_decode_workspace_size")
    return n.value


def _stream_handle(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _req(t, name, dtype, shape, device):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device.type != "cuda" or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on {device or 'a CUDA device'}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.data_ptr() % 16:
        raise ValueError(f"{name} must be 16-byte aligned")


@dataclass
class Plan:
    """A split-KV schedule in a device workspace (valid for one seq_lens)."""
    batch: int
    s_q: int
    max_pages: int
    workspace: object   # torch.uint8 CUDA tensor, owned by this Plan
    seq_lens: object    # the device seq_lens it was built from
    home: object = None  # handle of the stream that plan() allocated the workspace on (None: the caller's own)

    def problem(self, flags: int = 0) -> _Problem:
        return _problem(self.batch, self.s_q, self.max_pages, flags)


def _used_on(workspace, home, stream):
    """The workspace that plan() allocated is about to be used on `stream` (a torch stream).

    The plan owns it and may be dropped while that work is still queued: unless its memory
    belongs to that stream already, the allocator is told, and gives it out again only after.
    (A caller's own workspace is the caller's to keep.)
    """
    if home is not None and stream.cuda_stream != home:
        workspace.record_stream(stream)


def plan(seq_lens, *, s_q: int, max_pages_per_seq: int, workspace=None, stream=None) -> Plan:
    """Build the split-KV schedule on the device (``mla_decode_plan``).

    decode may run on another stream than the plan, ordered after it by an event; the plan may
    be dropped as soon as its last decode is enqueued.
    """
    import torch
    _req(seq_lens, "seq_lens", torch.int32, None, None)
    if seq_lens.dim() != 1:
        raise ValueError("seq_lens must be 1-D [batch]")
    batch = seq_lens.shape[0]
    with torch.cuda.device(seq_lens.device):
        need = workspace_size(batch, s_q, max_pages_per_seq)
        s = torch.cuda.current_stream() if stream is None else stream
        home = None
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=seq_lens.device)
            home = s.cuda_stream if stream is None else torch.cuda.current_stream().cuda_stream
        _req(workspace, "workspace", torch.uint8, None, seq_lens.device)
        prob = _problem(batch, s_q, max_pages_per_seq)
        _used_on(workspace, home, s)
        _check(load_library().mla_decode_plan(ctypes.byref(prob), seq_lens.data_ptr(),
                                              workspace.data_ptr(), workspace.numel(),
                                              _stream_handle(s)), "mla_decode_plan")
    return Plan(batch, s_q, max_pages_per_seq, workspace, seq_lens, home)


def decode(p: Plan, q_latent, q_rope, kv_cache, block_table, *, scale: float = DEFAULT_SCALE,
           out=None, lse=None, stream=None, events=None, pow2_max: bool = False):
    """Weight-absorbed MLA decode (``mla_decode``) -> (o_latent bf16, lse fp32).

    events: optional three torch.cuda.Event(enable_timing=True) recorded before the
    main kernel, between the main kernel and the merge, and after the merge
    (``mla_decode_timed``).  pow2_max: power-of-two running maxima
    (MLA_FLAG_POW2_MAX), so that every rescale is by an exact power of two.
    """
    return _decode(p, q_latent, q_rope, kv_cache, block_table, scale, out, lse, stream, events, None,
                   MLA_FLAG_POW2_MAX if pow2_max else 0)


def decode_fp8(p: Plan, q_latent, q_rope, kv_cache_fp8, block_table, *, scale: float = DEFAULT_SCALE,
               out=None, lse=None, stream=None, events=None, pow2_max: bool = False):
    """``mla_decode_fp8``: decode over an fp8 cache (uint8 [num_pages][64][656]) -> (o bf16, lse fp32).

    events and pow2_max as in ``decode``.
    """
    return _decode(p, q_latent, q_rope, kv_cache_fp8, block_table, scale, out, lse, stream, events, None,
                   MLA_FLAG_POW2_MAX if pow2_max else 0, fp8=True)


MLA_INJECT_WITHHOLD_K_LOAD = 0x1


def decode_diag(p: Plan, q_latent, q_rope, kv_cache, block_table, *, wait_limit_ns: int,
                inject: int = 0, scale: float = DEFAULT_SCALE, out=None, lse=None, stream=None):
    """``mla_decode_diag``: decode with a chosen wait limit and an optional injected stall.

    With inject=MLA_INJECT_WITHHOLD_K_LOAD one K-stage load of the unit that runs the
    schedule's first item is never issued, so the kernel's bounded waits run out: check(p) then reports
    MLA_DEV_TIMEOUT and the rows of that unit are unspecified.
    """
    return _decode(p, q_latent, q_rope, kv_cache, block_table, scale, out, lse, stream, None,
                   (int(wait_limit_ns), int(inject)), 0)


def _decode(p, q_latent, q_rope, kv_cache, block_table, scale, out, lse, stream, events, diag, flags,
            fp8=False):
    import torch
    dev = p.workspace.device
    B, S = p.batch, p.s_q
    _req(q_latent, "q_latent", torch.bfloat16, (B, S, NUM_HEADS, D_LATENT), dev)
    _req(q_rope, "q_rope", torch.bfloat16, (B, S, NUM_HEADS, D_ROPE), dev)
    if fp8:
        _req(kv_cache, "kv_cache_fp8", torch.uint8, None, dev)
        if kv_cache.dim() != 3 or tuple(kv_cache.shape[1:]) != (PAGE_SIZE, FP8_ROW_BYTES):
            raise ValueError("kv_cache_fp8 must be [num_pages][64][656] bytes")
    else:
        _req(kv_cache, "kv_cache", torch.bfloat16, None, dev)
        if kv_cache.dim() != 3 or tuple(kv_cache.shape[1:]) != (PAGE_SIZE, D_LATENT + D_ROPE):
            raise ValueError("kv_cache must be [num_pages][64][576]")
    _req(block_table, "block_table", torch.int32, (B, p.max_pages), dev)
    if out is None:
        out = torch.empty((B, S, NUM_HEADS, D_LATENT), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, S, NUM_HEADS), dtype=torch.float32, device=dev)
    _req(out, "out", torch.bfloat16, (B, S, NUM_HEADS, D_LATENT), dev)
    _req(lse, "lse", torch.float32, (B, S, NUM_HEADS), dev)
    prob = p.problem(flags)
    s = torch.cuda.current_stream() if stream is None else stream
    _used_on(p.workspace, p.home, s)
    args = [ctypes.byref(prob), q_latent.data_ptr(), q_rope.data_ptr(), kv_cache.data_ptr(),
            kv_cache.shape[0], block_table.data_ptr(), float(scale), out.data_ptr(),
            lse.data_ptr(), p.workspace.data_ptr(), p.workspace.numel(), _stream_handle(s)]
    handles = None
    if events is not None:
        if len(events) != 3:
            raise ValueError("events must hold three torch.cuda.Event")
        handles = (ctypes.c_void_p * 3)(*[ctypes.c_void_p(e.cuda_event) if e is not None
                                          else None for e in events])
    with torch.cuda.device(dev):
        if fp8:
            _check(load_library().mla_decode_fp8(*args, handles), "mla_decode_fp8")
        elif diag is not None:
            _check(load_library().mla_decode_diag(*args, *diag), "mla_decode_diag")
        elif handles is None:
            _check(load_library().mla_decode(*args), "mla_decode")
        else:
            _check(load_library().mla_decode_timed(*args, handles), "mla_decode_timed")
    return out, lse


NOALLOC_SCRATCH_BYTES = 64 << 20


def decode_noalloc(q_latent, q_rope, kv_cache, block_table, seq_lens, *, s_q: int,
                   scale: float = DEFAULT_SCALE, out=None, lse=None, stream=None):
    """Plan + decode through ``mla_decode_noalloc``: the library allocates nothing.

    For callers that cannot allocate device memory on their decode path; the
    workspace lives in a fixed 64 MiB device array inside the library, shared
    by every call (order calls on one stream).  Problems needing a larger
    workspace raise MLAError (status 3).  out / lse may be passed in so that
    this call allocates nothing on the Python side either.
    """
    import torch
    _req(seq_lens, "seq_lens", torch.int32, None, None)
    dev = seq_lens.device
    B = seq_lens.shape[0]
    _req(q_latent, "q_latent", torch.bfloat16, (B, s_q, NUM_HEADS, D_LATENT), dev)
    _req(q_rope, "q_rope", torch.bfloat16, (B, s_q, NUM_HEADS, D_ROPE), dev)
    _req(kv_cache, "kv_cache", torch.bfloat16, None, dev)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [batch][max_pages_per_seq]")
    _req(block_table, "block_table", torch.int32, None, dev)
    if out is None:
        out = torch.empty((B, s_q, NUM_HEADS, D_LATENT), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, s_q, NUM_HEADS), dtype=torch.float32, device=dev)
    _req(out, "out", torch.bfloat16, (B, s_q, NUM_HEADS, D_LATENT), dev)
    _req(lse, "lse", torch.float32, (B, s_q, NUM_HEADS), dev)
    prob = _problem(B, s_q, block_table.shape[1])
    with torch.cuda.device(dev):
        _check(load_library().mla_decode_noalloc(
            ctypes.byref(prob), q_latent.data_ptr(), q_rope.data_ptr(), kv_cache.data_ptr(),
            kv_cache.shape[0], block_table.data_ptr(), seq_lens.data_ptr(), float(scale),
            out.data_ptr(), lse.data_ptr(), _stream_handle(stream)), "mla_decode_noalloc")
    return out, lse


D_NOPE = 128
DEFAULT_ROPE_BASE = 10000.0
DEFAULT_RMS_EPS = 1e-6


ROPE_TABLE_FLOATS = 64
_rope_tables = {}


def rope_table(rope_base: float = DEFAULT_ROPE_BASE, device=None, stream=None):
    """The rotary table of ``mla_prolog_rope_table`` (float32 [64] on the device), built on the GPU."""
    import torch
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        table = torch.empty(ROPE_TABLE_FLOATS, dtype=torch.float32, device=dev)
        _check(load_library().mla_prolog_rope_table(float(rope_base), table.data_ptr(),
                                                    _stream_handle(stream)), "mla_prolog_rope_table")
    return table


def prolog(q_nope, q_pe, kv_latent, k_pe, w_uk, kv_norm_weight, kv_cache, block_table, seq_lens, *,
           rope_base: float = DEFAULT_ROPE_BASE, rms_eps: float = DEFAULT_RMS_EPS, table=None,
           q_latent=None, q_rope=None, status=None, stream=None):
    """The MLA prolog slice (``mla_prolog``): absorbed query, RoPE, cache append.

    Shapes: q_nope [B][s_q][128][128], q_pe [B][s_q][128][64], kv_latent [B][s_q][512],
    k_pe [B][s_q][64], w_uk [128][128][512], kv_norm_weight [512] (all bf16);
    kv_cache [pages][64][576] bf16 is updated in place; block_table [B][max_pages]
    and seq_lens [B] int32.  table: a rope_table() tensor; without one, the table of
    rope_base is built once per device and kept.  Returns (q_latent, q_rope, status):
    status is a one-element int32 device tensor of MLA_DEV_* bits (zeroed here, on the
    stream, unless the caller passes its own).
    """
    import torch
    if q_nope.dim() != 4:
        raise ValueError("q_nope must be [batch][s_q][heads][128]")
    B, S = q_nope.shape[0], q_nope.shape[1]
    dev = q_nope.device
    _req(q_nope, "q_nope", torch.bfloat16, (B, S, NUM_HEADS, D_NOPE), dev)
    _req(q_pe, "q_pe", torch.bfloat16, (B, S, NUM_HEADS, D_ROPE), dev)
    _req(kv_latent, "kv_latent", torch.bfloat16, (B, S, D_LATENT), dev)
    _req(k_pe, "k_pe", torch.bfloat16, (B, S, D_ROPE), dev)
    _req(w_uk, "w_uk", torch.bfloat16, (NUM_HEADS, D_NOPE, D_LATENT), dev)
    _req(kv_norm_weight, "kv_norm_weight", torch.bfloat16, (D_LATENT,), dev)
    _req(kv_cache, "kv_cache", torch.bfloat16, None, dev)
    if kv_cache.dim() != 3 or tuple(kv_cache.shape[1:]) != (PAGE_SIZE, D_LATENT + D_ROPE):
        raise ValueError("kv_cache must be [num_pages][64][576]")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [batch][max_pages_per_seq]")
    _req(block_table, "block_table", torch.int32, None, dev)
    _req(seq_lens, "seq_lens", torch.int32, (B,), dev)
    if q_latent is None:
        q_latent = torch.empty((B, S, NUM_HEADS, D_LATENT), dtype=torch.bfloat16, device=dev)
    if q_rope is None:
        q_rope = torch.empty((B, S, NUM_HEADS, D_ROPE), dtype=torch.bfloat16, device=dev)
    _req(q_latent, "q_latent", torch.bfloat16, (B, S, NUM_HEADS, D_LATENT), dev)
    _req(q_rope, "q_rope", torch.bfloat16, (B, S, NUM_HEADS, D_ROPE), dev)
    with torch.cuda.device(dev):
        if table is None:
            key = (dev.index, float(rope_base))
            table = _rope_tables.get(key)
            if table is None:
                # the kept table must hold its values for every later call on any stream
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("prolog: build the rotary table with rope_table() before "
                                       "capturing a CUDA graph, and pass it as table=")
                table = rope_table(rope_base, dev, stream)
                (stream if stream is not None else torch.cuda.current_stream()).synchronize()
                _rope_tables[key] = table
        _req(table, "table", torch.float32, (ROPE_TABLE_FLOATS,), dev)
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=dev)
        _req(status, "status", torch.int32, (1,), dev)
        prob = _problem(B, S, block_table.shape[1])
        _check(load_library().mla_prolog(
            ctypes.byref(prob), q_nope.data_ptr(), q_pe.data_ptr(), kv_latent.data_ptr(),
            k_pe.data_ptr(), w_uk.data_ptr(), kv_norm_weight.data_ptr(), float(rms_eps),
            table.data_ptr(), kv_cache.data_ptr(), kv_cache.shape[0], block_table.data_ptr(),
            seq_lens.data_ptr(), q_latent.data_ptr(), q_rope.data_ptr(), status.data_ptr(),
            _stream_handle(stream)), "mla_prolog")
    return q_latent, q_rope, status


D_V = 128
HIDDEN = 7168


def epilog_uv(o_latent, w_uv, *, o_v=None, status=None, stream=None):
    """The value up-projection (``mla_epilog_uv``): o_v[t][h] = W_UV[h] . o_latent[t][h].

    o_latent [B][s_q][128][512] and w_uv [128][128][512] bf16 -> (o_v [B][s_q][128][128] bf16,
    status: one-element int32 device tensor of MLA_DEV_* bits).
    """
    import torch
    if o_latent.dim() != 4:
        raise ValueError("o_latent must be [batch][s_q][heads][512]")
    B, S = o_latent.shape[0], o_latent.shape[1]
    dev = o_latent.device
    _req(o_latent, "o_latent", torch.bfloat16, (B, S, NUM_HEADS, D_LATENT), dev)
    _req(w_uv, "w_uv", torch.bfloat16, (NUM_HEADS, D_V, D_LATENT), dev)
    if o_v is None:
        o_v = torch.empty((B, S, NUM_HEADS, D_V), dtype=torch.bfloat16, device=dev)
    _req(o_v, "o_v", torch.bfloat16, (B, S, NUM_HEADS, D_V), dev)
    with torch.cuda.device(dev):
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=dev)
        _req(status, "status", torch.int32, (1,), dev)
        prob = _problem(B, S, 1)
        _check(load_library().mla_epilog_uv(ctypes.byref(prob), o_latent.data_ptr(), w_uv.data_ptr(),
                                            o_v.data_ptr(), status.data_ptr(), _stream_handle(stream)),
               "mla_epilog_uv")
    return o_v, status


def epilog_oproj(o_v, w_o, *, out=None, status=None, stream=None):
    """The output projection (``mla_epilog_oproj``, a tensor-core kernel): out = o_v . W_O^T.

    o_v [..][128][128] bf16 viewed as [tokens][16384], w_o [hidden][16384] bf16 ->
    out [tokens][hidden] bf16.  status: optional int32 device tensor of one element that
    the call ORs MLA_DEV_TIMEOUT into if a bounded wait in the kernel runs out.
    """
    import torch
    dev = o_v.device
    tokens = o_v.numel() // (NUM_HEADS * D_V)
    if tokens * NUM_HEADS * D_V != o_v.numel() or tokens < 1:
        raise ValueError("o_v must hold whole [128][128] token rows")
    _req(o_v, "o_v", torch.bfloat16, None, dev)
    if w_o.dim() != 2 or w_o.shape[1] != NUM_HEADS * D_V:
        raise ValueError("w_o must be [hidden][16384]")
    _req(w_o, "w_o", torch.bfloat16, None, dev)
    hidden = w_o.shape[0]
    if out is None:
        out = torch.empty((tokens, hidden), dtype=torch.bfloat16, device=dev)
    _req(out, "out", torch.bfloat16, (tokens, hidden), dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    _req(status, "status", torch.int32, None, dev)
    with torch.cuda.device(dev):
        _check(load_library().mla_epilog_oproj(int(tokens), int(hidden), o_v.data_ptr(), w_o.data_ptr(),
                                               out.data_ptr(), status.data_ptr(), _stream_handle(stream)),
               "mla_epilog_oproj")
    return out


FP8_ROW_BYTES = 656


def quantize_cache_fp8(kv_cache, *, out=None, stream=None):
    """The fp8 (e4m3) cache of a bf16 cache (``mla_cache_quantize_fp8``).

    kv_cache [..][576] bf16 -> uint8 [..][656]: per row the 512 e4m3 codes of c_kv / s,
    k_rope / s (bf16), s (fp32), zero padding.
    """
    import torch
    if kv_cache.shape[-1] != D_LATENT + D_ROPE:
        raise ValueError("kv_cache rows must hold 576 values")
    _req(kv_cache, "kv_cache", torch.bfloat16, None, None)
    dev = kv_cache.device
    shape = tuple(kv_cache.shape[:-1]) + (FP8_ROW_BYTES,)
    if out is None:
        out = torch.empty(shape, dtype=torch.uint8, device=dev)
    _req(out, "out", torch.uint8, shape, dev)
    rows = kv_cache.numel() // (D_LATENT + D_ROPE)
    with torch.cuda.device(dev):
        _check(load_library().mla_cache_quantize_fp8(kv_cache.data_ptr(), int(rows), out.data_ptr(),
                                                     _stream_handle(stream)), "mla_cache_quantize_fp8")
    return out


# ----------------------------------------------------------------------------- trees of drafted tokens

TREE_MAX_NODES = 64
MLA_DEV_BAD_OFFSETS = 0x10
MLA_DEV_BAD_PATH = 0x20


_host = None
_HOST_ENTRIES = ("mla_query", "mla_cache_append", "mla_cache_append_fp8", "mla_tree_workspace_size", "mla_tree_plan",
                 "mla_tree_decode", "mla_tree_decode_fp8", "mla_cache_commit")


class _PythonOnly:
    """Stands for the native marshalling where there is none: no call is the plain case."""

    query = append = tree_plan = tree_decode = commit = staticmethod(lambda *a: None)


def _native():
    """The marshalling of the tree step's calls in C++ (csrc/host/mla_host.cpp).

    Its functions take the plain case, dense CUDA tensors on the current device and stream, and
    return None for any other; the Python below then does the call or says what is wrong with it.
    Without the module the Python does every call, 10-25 us slower each.
    """
    global _host
    if _host is None:
        lib = load_library()
        try:
            module = _load_host()
        except ImportError as e:
            warnings.warn(f"calls are marshalled in Python: {e} (python -m mla_decode_attention_02_gb300.build)",
                          stacklevel=3)
            _host = _PythonOnly
            return _host
        module.bind(*[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _HOST_ENTRIES])
        _host = module
    return _host


def _load_host():
    """The host module built for this Python and this torch; ImportError if there is none."""
    import importlib.machinery
    import importlib.util

    import torch  # noqa: F401  (its libraries are what the module links to)

    from .build import host_path
    path = host_path()
    if not os.path.exists(path):
        raise ImportError(f"{os.path.basename(path)} is missing")
    name = __package__ + "._mla_host"
    spec = importlib.util.spec_from_file_location(name, path,
                                                  loader=importlib.machinery.ExtensionFileLoader(name, path))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _made(r, what):
    """The outputs of a native call, or the error of one that the C ABI refused."""
    if type(r) is int:
        raise MLAError(r, what)
    return r


def _kept_table(table, t, rope_base):
    """The caller's table, or the kept one of rope_base if there is one."""
    if table is not None:
        return table
    return _rope_tables.get((t.get_device(), float(rope_base))) if hasattr(t, "get_device") else None


def _launch_on(index, stream, *tensors):
    """Context of a call: its device, and its stream as the current one, so that what the call
    allocates or clears belongs to that stream too.  On a stream of the caller's choice the
    tensors are marked as in use there, so that freeing one does not hand its memory out early."""
    import torch
    if stream is None:
        return _HERE_ALREADY if torch.cuda.current_device() == index else torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"stream must be one of cuda:{index}, the tensors' device")
    for t in tensors:   # (what is no CUDA tensor is refused, or not looked at, later)
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


_HERE_ALREADY = contextlib.nullcontext()


def _current_stream(index) -> int:
    """Handle of the current stream of a device (a few times cheaper than a torch.cuda.Stream object: a
    small operator's launch takes a few microseconds in all)."""
    import torch
    return torch._C._cuda_getCurrentRawStream(index)


def _ragged(batch: int, tokens: int, max_pages: int, flags: int = 0) -> _Ragged:
    return _Ragged(int(batch), int(tokens), NUM_HEADS, PAGE_SIZE, int(max_pages), int(flags))


def _refuse(t, name, dtype, shape, index, strided=False):
    """Raise what is wrong with an argument that _dense or _strided did not take."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not strided and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be 16-byte aligned (integers: to their size)")


def _dense(t, name, dtype, shape, index, align=16) -> int:
    """Address of a dense array of this dtype and shape on device `index`.

    A call of a small operator takes a few microseconds on the GPU, so what is not needed to
    accept an argument is left to _refuse.
    """
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            ptr = t.data_ptr()
            if not ptr % align:
                return ptr
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, index)


def _strided(t, name, dtype, shape, index):
    """Address and strides (in elements) of an input whose last dim is contiguous.

    The others may be strided (a view of a larger projection): positive multiples of 8.
    """
    try:
        ptr = t.data_ptr()
        taken = t.dtype is dtype and t.shape == shape and t.get_device() == index and not ptr % 16
    except AttributeError:
        taken = False
    if not taken:
        _refuse(t, name, dtype, shape, index, strided=True)
    st = t.stride()
    if st[-1] != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    # the stride of a dimension of one element is never used: any legal value does
    if shape[0] == 1:
        st = (8,) + st[1:]
    for v in st[:-1]:
        if v < 1 or v % 8 or v >= 1 << 31:
            raise ValueError(f"{name}'s strides must be positive multiples of 8")
    return (ptr, *st[:-1])


def _index_of(t, name, dim, dtype) -> int:
    """Device index of the argument that fixes the device and a size, with its dimension count."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != dim or 0 in shape:
        raise ValueError(f"{name} must have {dim} non-empty dimensions, got {tuple(shape)}")
    index = t.get_device()
    if index < 0:
        _refuse(t, name, dtype, shape, index)
    return index


def _out(t, name, dtype, shape, index):
    """The caller's output, or a new one on the current stream."""
    import torch
    if t is None:
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", index))
    _dense(t, name, dtype, shape, index, 4 if dtype is torch.int32 else 16)
    return t


def _bytes(t, name, index):
    """Address and size of the caller's bytes, of any shape."""
    import torch
    return _dense(t, name, torch.uint8, getattr(t, "shape", None), index), t.numel()


def _status_word(status, index):
    import torch
    if status is None:
        return torch.zeros(1, dtype=torch.int32, device=torch.device("cuda", index))
    _dense(status, "status", torch.int32, (1,), index, 4)
    return status


def _table_of(table, rope_base, index, what) -> int:
    """Address of the caller's table, or of rope_base's, built once per device and kept (call on the launch's stream)."""
    import torch
    if table is None:
        key = (index, float(rope_base))
        table = _rope_tables.get(key)
        if table is None:
            # the kept table must hold its values for every later call on any stream
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError(f"{what}: build the rotary table with rope_table() before "
                                   "capturing a CUDA graph, and pass it as table=")
            table = rope_table(rope_base, torch.device("cuda", index))
            torch.cuda.current_stream().synchronize()
            _rope_tables[key] = table
    return _dense(table, "table", torch.float32, (ROPE_TABLE_FLOATS,), index, 4)


def _cache_ptr(kv_cache, fp8, index, layers=False) -> int:
    import torch
    name, dtype, row = (("kv_cache_fp8", torch.uint8, FP8_ROW_BYTES) if fp8 else
                        ("kv_cache", torch.bfloat16, D_LATENT + D_ROPE))
    if not isinstance(kv_cache, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = kv_cache.shape
    if shape[-2:] != (PAGE_SIZE, row) or not (len(shape) == 3 or (layers and len(shape) == 4)) or 0 in shape:
        if kv_cache.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {kv_cache.dtype}")
        raise ValueError(f"{name} must be {'([layers])' if layers else ''}[num_pages][64][{row}]")
    return _dense(kv_cache, name, dtype, shape, index)


def query(q_nope, q_pe, w_uk, positions, *, rope_base: float = DEFAULT_ROPE_BASE, table=None, q_latent=None,
          q_rope=None, status=None, stream=None):
    """Absorbed and rotated queries at explicit positions (``mla_query``).

    q_nope [T][128][128] and q_pe [T][128][64] bf16 (last dim contiguous, otherwise strided:
    both may be views of one projection's output), w_uk [128][128][512] bf16, positions [T]
    int32; a negative position leaves the token's output rows as they were.  table: a
    rope_table() tensor; without one, the table of rope_base is built once per device and
    kept.  Returns (q_latent [T][128][512], q_rope [T][128][64], status): status is a
    one-element int32 device tensor of MLA_DEV_* bits.
    """
    if stream is None:
        r = (_host or _native()).query(q_nope, q_pe, w_uk, positions, _kept_table(table, q_nope, rope_base), q_latent,
                                       q_rope, status)
        if r is not None:
            return _made(r, "mla_query")
    import torch
    index = _index_of(q_nope, "q_nope", 3, torch.bfloat16)
    T = q_nope.shape[0]
    args = (*_strided(q_nope, "q_nope", torch.bfloat16, (T, NUM_HEADS, D_NOPE), index),
            *_strided(q_pe, "q_pe", torch.bfloat16, (T, NUM_HEADS, D_ROPE), index),
            _dense(w_uk, "w_uk", torch.bfloat16, (NUM_HEADS, D_NOPE, D_LATENT), index))
    pos = _dense(positions, "positions", torch.int32, (T,), index, 4)
    with _launch_on(index, stream, q_nope, q_pe, w_uk, positions, table, q_latent, q_rope, status):
        tab = _table_of(table, rope_base, index, "query")
        q_latent = _out(q_latent, "q_latent", torch.bfloat16, (T, NUM_HEADS, D_LATENT), index)
        q_rope = _out(q_rope, "q_rope", torch.bfloat16, (T, NUM_HEADS, D_ROPE), index)
        status = _status_word(status, index)
        _check(load_library().mla_query(T, *args, tab, pos, q_latent.data_ptr(), q_rope.data_ptr(), status.data_ptr(),
                                        _current_stream(index)), "mla_query")
    return q_latent, q_rope, status


def cache_append(kv_latent, k_pe, kv_norm_weight, kv_cache, block_table, seq_lens, token_offsets, *, positions=None,
                 rope_base: float = DEFAULT_ROPE_BASE, rms_eps: float = DEFAULT_RMS_EPS, table=None, status=None,
                 stream=None):
    """Append ragged tokens to the paged cache (``mla_cache_append``) -> status.

    kv_latent [T][512] (before RMSNorm) and k_pe [T][64] (before RoPE) bf16, last dim contiguous,
    rows strided at will; kv_norm_weight [512] bf16; kv_cache [pages][64][576] bf16, updated in
    place; block_table [B][max_pages], seq_lens [B] (these tokens counted) and token_offsets
    [B + 1] int32: request b's tokens are rows token_offsets[b] .. token_offsets[b + 1] - 1 and
    go to its last slots.  positions [T] int32: RoPE positions (default: the slots); a negative
    one leaves the token out.  table, status as in ``query``.
    """
    return _append(kv_latent, k_pe, kv_norm_weight, kv_cache, block_table, seq_lens, token_offsets, positions,
                   rope_base, rms_eps, table, status, stream, False)


def cache_append_fp8(kv_latent, k_pe, kv_norm_weight, kv_cache_fp8, block_table, seq_lens, token_offsets, *,
                     positions=None, rope_base: float = DEFAULT_ROPE_BASE, rms_eps: float = DEFAULT_RMS_EPS,
                     table=None, status=None, stream=None):
    """``cache_append`` into an fp8 cache (``mla_cache_append_fp8``; uint8 [pages][64][656])."""
    return _append(kv_latent, k_pe, kv_norm_weight, kv_cache_fp8, block_table, seq_lens, token_offsets, positions,
                   rope_base, rms_eps, table, status, stream, True)


def _append(kv_latent, k_pe, kv_norm_weight, kv_cache, block_table, seq_lens, token_offsets, positions, rope_base,
            rms_eps, table, status, stream, fp8):
    if stream is None:
        r = (_host or _native()).append(fp8, kv_latent, k_pe, kv_norm_weight, kv_cache, block_table, seq_lens,
                                        token_offsets, positions, rms_eps, _kept_table(table, kv_latent, rope_base),
                                        status)
        if r is not None:
            return _made(r, "mla_cache_append_fp8" if fp8 else "mla_cache_append")
    import torch
    index = _index_of(kv_latent, "kv_latent", 2, torch.bfloat16)
    T = kv_latent.shape[0]
    lat = _strided(kv_latent, "kv_latent", torch.bfloat16, (T, D_LATENT), index)
    pe = _strided(k_pe, "k_pe", torch.bfloat16, (T, D_ROPE), index)
    gamma = _dense(kv_norm_weight, "kv_norm_weight", torch.bfloat16, (D_LATENT,), index)
    cache = _cache_ptr(kv_cache, fp8, index)
    _index_of(block_table, "block_table", 2, torch.int32)
    B, width = block_table.shape
    bt = _dense(block_table, "block_table", torch.int32, (B, width), index, 4)
    sl = _dense(seq_lens, "seq_lens", torch.int32, (B,), index, 4)
    off = _dense(token_offsets, "token_offsets", torch.int32, (B + 1,), index, 4)
    pos = None if positions is None else _dense(positions, "positions", torch.int32, (T,), index, 4)
    lib = load_library()
    with _launch_on(index, stream, kv_latent, k_pe, kv_norm_weight, kv_cache, block_table, seq_lens, token_offsets,
                    positions, table, status):
        tab = _table_of(table, rope_base, index, "cache_append")
        status = _status_word(status, index)
        prob = _Ragged(B, T, NUM_HEADS, PAGE_SIZE, width, 0)
        f = lib.mla_cache_append_fp8 if fp8 else lib.mla_cache_append
        _check(f(ctypes.byref(prob), *lat, *pe, gamma, float(rms_eps), tab, pos, cache, kv_cache.shape[0], bt, sl, off,
                 status.data_ptr(), _current_stream(index)),
               "mla_cache_append_fp8" if fp8 else "mla_cache_append")
    return status


@dataclass
class TreePlan:
    """A split-KV schedule of a batch of trees in a device workspace (one step's lengths, offsets and masks)."""
    batch: int
    tokens: int
    max_pages: int
    workspace: object   # torch.uint8 CUDA tensor, owned by this TreePlan
    scratch_fits: bool = True   # until a tree_decode_fp8 finds no memory for its own scratch

    def problem(self, flags: int = 0) -> _Ragged:
        return _ragged(self.batch, self.tokens, self.max_pages, flags)


def tree_workspace_size(batch: int, tokens: int, max_pages: int) -> int:
    n = ctypes.c_size_t(0)
    prob = _ragged(batch, tokens, max_pages)
    _check(load_library().mla_tree_workspace_size(ctypes.byref(prob), ctypes.byref(n)), "mla_tree_workspace_size")
    return n.value


def tree_plan(seq_lens, token_offsets, masks, *, max_pages_per_seq: int, workspace=None, stream=None) -> TreePlan:
    """Build the schedule of a batch of drafted trees on the device (``mla_tree_plan``).

    seq_lens [B] int32 (cached keys, the trees' nodes included), token_offsets [B + 1] int32 (request
    b's nodes are rows token_offsets[b] .. token_offsets[b + 1] - 1 of the token arrays; at most
    64 each), masks [T] int64: bit j of a node's mask is set if it sees node j of its tree.  T may
    exceed token_offsets[B] (padding).  The plan serves every layer of the step; calls that share
    it must be ordered (by one stream, or events), and it may be dropped once the last is enqueued.
    """
    if stream is None:
        r = (_host or _native()).tree_plan(seq_lens, token_offsets, masks, max_pages_per_seq, workspace)
        if r is not None:
            return TreePlan(seq_lens.shape[0], masks.shape[0], max_pages_per_seq, _made(r, "mla_tree_plan"))
    import torch
    index = _index_of(seq_lens, "seq_lens", 1, torch.int32)
    B = seq_lens.shape[0]
    sl = _dense(seq_lens, "seq_lens", torch.int32, (B,), index, 4)
    off = _dense(token_offsets, "token_offsets", torch.int32, (B + 1,), index, 4)
    _index_of(masks, "masks", 1, torch.int64)
    T = masks.shape[0]
    m = _dense(masks, "masks", torch.int64, (T,), index, 8)
    lib = load_library()
    with _launch_on(index, stream, seq_lens, token_offsets, masks, workspace):
        prob = _ragged(B, T, max_pages_per_seq)
        if workspace is None:
            n = ctypes.c_size_t(0)
            _check(lib.mla_tree_workspace_size(ctypes.byref(prob), ctypes.byref(n)), "mla_tree_workspace_size")
            workspace = torch.empty(n.value, dtype=torch.uint8, device=seq_lens.device)
        ws, nbytes = _bytes(workspace, "workspace", index)
        workspace.record_stream(torch.cuda.current_stream())   # (the plan's, however it was made)
        _check(lib.mla_tree_plan(ctypes.byref(prob), sl, off, m, ws, nbytes, _current_stream(index)), "mla_tree_plan")
    return TreePlan(B, T, int(max_pages_per_seq), workspace)


def tree_decode(p: TreePlan, q_latent, q_rope, kv_cache, block_table, *, scale: float = DEFAULT_SCALE, out=None,
                lse=None, stream=None, pow2_max: bool = False):
    """Attention of drafted trees over the paged cache (``mla_tree_decode``) -> (o_latent bf16, lse fp32).

    q_latent [T][128][512], q_rope [T][128][64] bf16; outputs [T][128][512] and [T][128].  A node
    that sees no key gives o = 0 and lse = -inf; rows behind the last request are not written.
    ``check(p)`` reads the status bits.  pow2_max as in ``decode``.

    The softmax weights are rounded to bf16 for their product with the rows, as in ``decode``:
    o is off by 2.4e-3 of its norm at most (200 keys; 2.0e-3 over 4000), its own rounding being
    1.66e-3.  By default a weight may be rounded twice, and one visible key gives o exactly;
    with pow2_max never twice (2.31e-3 over 200 keys), but one key gives 1.5e-3.
    """
    return _tree_decode(p, q_latent, q_rope, kv_cache, block_table, scale, out, lse, stream, pow2_max, False)


def tree_decode_fp8(p: TreePlan, q_latent, q_rope, kv_cache_fp8, block_table, *, scale: float = DEFAULT_SCALE,
                    out=None, lse=None, stream=None, pow2_max: bool = True, scratch=None):
    """``tree_decode`` over an fp8 cache (``mla_tree_decode_fp8``; uint8 [pages][64][656]).

    pow2_max is on here: a weight times its token's scale is never exactly 1, so the exact
    running maximum gains nothing, and rescaling a page half to the pair's maximum by a power
    of two does not round its weights a second time (error of o over 100-200 keys 2.45e-3 ->
    2.32e-3 of its norm, 1.66e-3 being its own rounding to bf16).

    scratch: where each page is expanded once for all nodes, a uint8 tensor of at least
    batch * max_pages * EXPANDED_PAGE_BYTES bytes, or False for none.  By default one is allocated
    for the call if the trees average two nodes or more and it takes no more than
    EXPAND_LIMIT_BYTES; where there is no memory for it, this and the plan's later calls go
    without.  The results are the same bit for bit.
    """
    return _tree_decode(p, q_latent, q_rope, kv_cache_fp8, block_table, scale, out, lse, stream, pow2_max, True,
                        scratch)


EXPANDED_PAGE_BYTES = PAGE_SIZE * (2 * (D_LATENT + D_ROPE) + 4)
EXPAND_LIMIT_BYTES = 8 << 30


def _tree_decode(p, q_latent, q_rope, kv_cache, block_table, scale, out, lse, stream, pow2_max, fp8, scratch=False):
    T, ws = p.tokens, p.workspace
    if fp8 and scratch is None:
        need = p.batch * p.max_pages * EXPANDED_PAGE_BYTES
        wanted = p.scratch_fits and T >= 2 * p.batch and need <= EXPAND_LIMIT_BYTES and p.batch <= 65535
        scratch = need if wanted else False
    elif scratch is not None and scratch is not False and not hasattr(scratch, "data_ptr"):
        raise TypeError("scratch must be a torch.Tensor, False or None")
    if stream is None:
        call = (_host or _native()).tree_decode
        args = (p.batch, T, p.max_pages, ws, q_latent, q_rope, kv_cache, block_table, scale, out, lse,
                MLA_FLAG_POW2_MAX if pow2_max else 0, fp8)
        r = call(*args, None if scratch is False else scratch)
        if r is False:      # no memory for the scratch
            p.scratch_fits = scratch = False
            r = call(*args, None)
        if r is not None:
            return _made(r, "mla_tree_decode_fp8" if fp8 else "mla_tree_decode")
    import torch
    index = ws.get_device()
    ql = _dense(q_latent, "q_latent", torch.bfloat16, (T, NUM_HEADS, D_LATENT), index)
    qr = _dense(q_rope, "q_rope", torch.bfloat16, (T, NUM_HEADS, D_ROPE), index)
    cache = _cache_ptr(kv_cache, fp8, index)
    bt = _dense(block_table, "block_table", torch.int32, (p.batch, p.max_pages), index, 4)
    lib = load_library()
    with _launch_on(index, stream, ws, q_latent, q_rope, kv_cache, block_table, out, lse, scratch):
        out = _out(out, "out", torch.bfloat16, (T, NUM_HEADS, D_LATENT), index)
        lse = _out(lse, "lse", torch.float32, (T, NUM_HEADS), index)
        ws.record_stream(torch.cuda.current_stream())
        prob = _Ragged(p.batch, T, NUM_HEADS, PAGE_SIZE, p.max_pages, MLA_FLAG_POW2_MAX if pow2_max else 0)
        args = (ctypes.byref(prob), ql, qr, cache, kv_cache.shape[0], bt, float(scale), out.data_ptr(), lse.data_ptr(),
                ws.data_ptr(), ws.numel())
        if not fp8:
            _check(lib.mla_tree_decode(*args, _current_stream(index)), "mla_tree_decode")
            return out, lse
        if scratch is not False and isinstance(scratch, int):
            try:
                scratch = torch.empty(scratch, dtype=torch.uint8, device=ws.device)
            except torch.OutOfMemoryError:
                p.scratch_fits = scratch = False
        room = (None, 0)
        if scratch is not False:
            room = _bytes(scratch, "scratch", index)
        _check(lib.mla_tree_decode_fp8(*args, *room, _current_stream(index)), "mla_tree_decode_fp8")
    return out, lse


def cache_commit(kv_cache, block_table, seq_lens, token_offsets, paths, path_lens, *, new_seq_lens=None, status=None,
                 stream=None):
    """Move the accepted nodes' rows to the front of their trees' slots (``mla_cache_commit``).

    kv_cache [pages][64][576] or [layers][pages][64][576] bf16, updated in place in every layer;
    paths [B][max_path] int32 (strictly increasing node indices, max_path <= 64), path_lens [B]
    int32; block_table, seq_lens and token_offsets as in ``cache_append``.  Returns
    (new_seq_lens [B] int32, status).
    """
    return _commit(kv_cache, block_table, seq_lens, token_offsets, paths, path_lens, new_seq_lens, status, stream,
                   False)


def cache_commit_fp8(kv_cache_fp8, block_table, seq_lens, token_offsets, paths, path_lens, *, new_seq_lens=None,
                     status=None, stream=None):
    """``cache_commit`` for fp8 caches (uint8 [pages][64][656] or [layers][pages][64][656])."""
    return _commit(kv_cache_fp8, block_table, seq_lens, token_offsets, paths, path_lens, new_seq_lens, status, stream,
                   True)


def _commit(kv_cache, block_table, seq_lens, token_offsets, paths, path_lens, new_seq_lens, status, stream, fp8):
    if stream is None:
        r = (_host or _native()).commit(fp8, kv_cache, block_table, seq_lens, token_offsets, paths, path_lens,
                                        new_seq_lens, status)
        if r is not None:
            return _made(r, "mla_cache_commit")
    import torch
    index = _index_of(block_table, "block_table", 2, torch.int32)
    B, width = block_table.shape
    bt = _dense(block_table, "block_table", torch.int32, (B, width), index, 4)
    cache = _cache_ptr(kv_cache, fp8, index, layers=True)
    sl = _dense(seq_lens, "seq_lens", torch.int32, (B,), index, 4)
    off = _dense(token_offsets, "token_offsets", torch.int32, (B + 1,), index, 4)
    _index_of(paths, "paths", 2, torch.int32)
    most = paths.shape[1]
    way = _dense(paths, "paths", torch.int32, (B, most), index, 4)
    lens = _dense(path_lens, "path_lens", torch.int32, (B,), index, 4)
    row = FP8_ROW_BYTES if fp8 else 2 * (D_LATENT + D_ROPE)
    shape = kv_cache.shape
    layers, pages = (shape[0] if len(shape) == 4 else 1), shape[-3]
    with _launch_on(index, stream, kv_cache, block_table, seq_lens, token_offsets, paths, path_lens, new_seq_lens,
                    status):
        new_seq_lens = _out(new_seq_lens, "new_seq_lens", torch.int32, (B,), index)
        status = _status_word(status, index)
        # the offsets alone say how many nodes there are: any bound on them will do
        prob = _Ragged(B, (1 << 24) - 1, NUM_HEADS, PAGE_SIZE, width, 0)
        _check(load_library().mla_cache_commit(
            ctypes.byref(prob), cache, layers, pages * PAGE_SIZE * row, row, pages, bt, sl, off, way, most, lens,
            new_seq_lens.data_ptr(), status.data_ptr(), _current_stream(index)), "mla_cache_commit")
    return new_seq_lens, status


def check(p, stream=None) -> int:
    """Synchronise and return the device status bits of a Plan or TreePlan (0 = no input error seen)."""
    import torch
    v = ctypes.c_int32(0)
    with torch.cuda.device(p.workspace.device):
        rc = load_library().mla_decode_check(p.workspace.data_ptr(), ctypes.byref(v),
                                             _stream_handle(stream))
    if rc not in (0, 5, 6):
        _check(rc, "mla_decode_check")
    return v.value


# ----------------------------------------------------------------------------- host planner

def _align(x: int, a: int) -> int:
    return (x + a - 1) // a * a


def plan_layout(batch: int, s_q: int, units: int, trees: int = 0) -> dict:
    """Byte offsets of the schedule regions (mirrors make_layout in csrc/mla_internal.h).

    A tree schedule has one row per token: batch * s_q is then the number of tokens, and trees its batch.
    """
    rows = batch * s_q
    max_items = rows + units
    off = 64
    L = {"num_rows": rows, "max_items": max_items, "items": off}
    off += 16 * max_items
    L["item_unit"] = off
    off += 4 * max_items
    L["unit_begin"] = off
    off += 4 * (units + 1)
    L["row_nparts"] = off
    off += 4 * rows
    L["row_part0"] = off
    off += 4 * rows
    L["row_item0"] = off
    off += 4 * rows
    off = _align(off, 8)
    L["row_pos"] = off
    off += 8 * rows
    if trees:
        off = _align(off, 16)
        L["tree_rows"] = off
        off += 16 * rows
        L["tree_items"] = off
        off += 16 * max_items
        L["tree_pages"] = off
        off += 4 * trees
    L["plan_end"] = off
    return L


_HDR = np.dtype([("magic", "<u4"), ("batch", "<i4"), ("s_q", "<i4"), ("max_pages", "<i4"),
                 ("num_units", "<i4"), ("num_rows", "<i4"), ("max_items", "<i4"),
                 ("num_items", "<i4"), ("num_parts", "<i4"), ("status", "<i4"),
                 ("split", "<i4"), ("min_split", "<i4"), ("total_cost", "<i8"),
                 ("target", "<i8")])


_TREE_ROW = np.dtype([("mask", "<u8"), ("context", "<i4"), ("req", "<i4")])


def parse_plan(buf, batch: int, s_q: int, units: int, trees: int = 0) -> dict:
    """Decode schedule bytes (host copy of a workspace prefix) into numpy arrays."""
    b = np.frombuffer(bytes(buf), dtype=np.uint8)
    L = plan_layout(batch, s_q, units, trees)
    hdr = b[:64].view(_HDR)[0]
    n = int(hdr["num_items"])
    R = L["num_rows"]
    items = b[L["items"]:L["items"] + 16 * n].view("<i4").reshape(n, 4)
    more = {"tree_rows": b[L["tree_rows"]:L["tree_rows"] + 16 * R].view(_TREE_ROW).copy(),
            "tree_items": b[L["tree_items"]:L["tree_items"] + 16 * n].view(_TREE_ROW).copy(),
            "tree_pages": b[L["tree_pages"]:L["tree_pages"] + 4 * trees].view("<i4").copy()} if trees else {}
    return {
        **more,
        "header": {k: int(hdr[k]) for k in _HDR.names},
        "items": items.copy(),   # columns: row, kv_begin, kv_end, part
        "item_unit": b[L["item_unit"]:L["item_unit"] + 4 * n].view("<i4").copy(),
        "unit_begin": b[L["unit_begin"]:L["unit_begin"] + 4 * (units + 1)].view("<i4").copy(),
        "row_nparts": b[L["row_nparts"]:L["row_nparts"] + 4 * R].view("<i4").copy(),
        "row_part0": b[L["row_part0"]:L["row_part0"] + 4 * R].view("<i4").copy(),
        "row_item0": b[L["row_item0"]:L["row_item0"] + 4 * R].view("<i4").copy(),
        "row_pos": b[L["row_pos"]:L["row_pos"] + 8 * R].view("<i8").copy(),
    }


def plan_host(seq_lens, *, s_q: int, max_pages_per_seq: int, num_units: int) -> dict:
    """Run the planner's algorithm on the CPU (``mla_decode_plan_host``) and parse it."""
    lib = load_library()
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    prob = _problem(sl.shape[0], s_q, max_pages_per_seq)
    nbytes = lib.mla_decode_plan_bytes(ctypes.byref(prob), int(num_units))
    if nbytes == 0:  # invalid problem: let the planner entry point name the reason
        _check(lib.mla_decode_plan_host(ctypes.byref(prob), sl.ctypes.data, int(num_units),
                                        None, 0), "mla_decode_plan_host")
        raise MLAError(1, "mla_decode_plan_bytes")
    buf = np.zeros(nbytes, dtype=np.uint8)
    _check(lib.mla_decode_plan_host(ctypes.byref(prob), sl.ctypes.data, int(num_units),
                                    buf.ctypes.data, nbytes), "mla_decode_plan_host")
    return parse_plan(buf.tobytes(), sl.shape[0], s_q, num_units)


def plan_device_bytes(p: Plan) -> bytes:
    """Host copy of a device schedule (for tests)."""
    L = plan_layout(p.batch, p.s_q, num_units())
    return p.workspace[:L["plan_end"]].cpu().numpy().tobytes()


def tree_plan_host(seq_lens, token_offsets, masks, *, max_pages_per_seq: int, num_units: int) -> dict:
    """Run the tree planner's algorithm on the CPU (``mla_tree_plan_host``) and parse it."""
    lib = load_library()
    sl, off = np.ascontiguousarray(seq_lens, np.int32), np.ascontiguousarray(token_offsets, np.int32)
    m = np.ascontiguousarray(masks, np.uint64)
    prob = _ragged(sl.shape[0], m.shape[0], max_pages_per_seq)
    nbytes = lib.mla_tree_plan_bytes(ctypes.byref(prob), int(num_units))
    buf = np.zeros(max(nbytes, 1), dtype=np.uint8)
    _check(lib.mla_tree_plan_host(ctypes.byref(prob), sl.ctypes.data, off.ctypes.data, m.ctypes.data, int(num_units),
                                  buf.ctypes.data, nbytes), "mla_tree_plan_host")
    return parse_plan(buf.tobytes(), 1, m.shape[0], num_units, trees=sl.shape[0])


def tree_plan_device(p: TreePlan) -> dict:
    """Host copy of a device schedule of trees, parsed (for tests)."""
    units = num_units()
    end = plan_layout(1, p.tokens, units, trees=p.batch)["plan_end"]
    return parse_plan(p.workspace[:end].cpu().numpy().tobytes(), 1, p.tokens, units, trees=p.batch)
