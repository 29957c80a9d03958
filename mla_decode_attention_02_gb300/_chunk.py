"""Binding of a layer step over chunks of prompts (include/mla_chunk.h): argument marshalling only.

Rotary positions of the chunk's queries, attention of its tokens over their requests' paged
caches, and the layer's boundary.  As in ``_binding``: tensors are checked, outputs and
workspaces made with PyTorch, pointers and the current stream passed through the C ABI.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass, field

from . import _binding as B
from ._binding import (D_LATENT, D_NOPE, D_ROPE, D_V, DEFAULT_RMS_EPS, DEFAULT_ROPE_BASE, DEFAULT_SCALE, NUM_HEADS,
                       PAGE_SIZE, _cache_ptr, _check, _current_stream, _dense, _index_of, _launch_on, _out, _SIGS,
                       _strided, load_library)

MLA_DEV_BAD_KV_TOKENS = 0x40


class _Chunk(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("flags", ctypes.c_int32), ("kv_tokens", ctypes.c_int64)]


_C = ctypes.POINTER(_Chunk)
_vp, _i32, _i64, _f32, _size = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_ATTEND = [_C, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _f32, _vp, _vp, _vp, _size, _vp, _size, _vp]
_SIGS.update({
    "mla_rope_table_scaled": (ctypes.c_int, [ctypes.c_double, _i32, ctypes.c_double, _i32, ctypes.c_double,
                                             ctypes.c_double, _vp, _vp]),
    "mla_rotate": (ctypes.c_int, [_i32, _i32, _i32, _vp, _i64, _i64, _vp, _vp, _i32, _i32, _f32, _vp, _i64, _i64, _vp]),
    "mla_residual_norm": (ctypes.c_int, [_i32, _i32, _vp, _i64, _vp, _i64, _vp, _f32, _vp, _vp, _vp]),
    "mla_residual_norm_fp8": (ctypes.c_int, [_i32, _i32, _vp, _i64, _vp, _i64, _vp, _f32, _i32, _vp, _vp, _vp, _vp]),
    "mla_chunk_workspace_size": (ctypes.c_int, [_C, ctypes.POINTER(_size)]),
    "mla_chunk_scratch_size": (ctypes.c_int, [_C, _i32, _i32, ctypes.POINTER(_size)]),
    "mla_chunk_plan": (ctypes.c_int, [_C, _vp, _vp, _vp, _size, _vp]),
    "mla_chunk_attend": (ctypes.c_int, _ATTEND),
    "mla_chunk_attend_fp8": (ctypes.c_int, _ATTEND),
})


def _int(v, name, bits=31) -> int:
    """An integer that the C ABI's field holds (ctypes would cut it to the field's bits)."""
    v = int(v)
    if not -1 << bits <= v < 1 << bits:
        raise ValueError(f"{name} must be below 2^{bits}, got {v}")
    return v


# ----------------------------------------------------------------------------- rotary positions

ROTARY_DIMS = (16, 32, 64, 128, 256)
_LAYOUTS = {"interleaved": 0, "half": 1}


def rope_table_scaled(rope_base: float = DEFAULT_ROPE_BASE, *, dims: int = D_ROPE, factor: float = 1.0,
                      original_positions: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None,
                      stream=None):
    """The rotary table of positions scaled for long contexts by YaRN (``mla_rope_table_scaled``): float32 [dims].

    Pairs that turn more than beta_fast times within original_positions keep their rate, those that turn
    less than beta_slow times are slowed by factor, those between are mixed.  With factor 1 it is
    ``rope_table``'s (for any dims).  For dims = 64 ``prolog``, ``query`` and ``cache_append`` take it as table=.
    """
    import torch
    if dims not in ROTARY_DIMS:
        raise ValueError(f"dims must be one of {ROTARY_DIMS}, got {dims}")
    original_positions = _int(original_positions, "original_positions")
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    index = torch.cuda.current_device() if dev.index is None else dev.index
    with _launch_on(index, stream):
        table = torch.empty(dims, dtype=torch.float32, device=torch.device("cuda", index))
        _check(load_library().mla_rope_table_scaled(float(rope_base), int(dims), float(factor), original_positions,
                                                    float(beta_fast), float(beta_slow), table.data_ptr(),
                                                    _current_stream(index)), "mla_rope_table_scaled")
    return table


def rotate(x, positions, *, table, layout: str = "interleaved", inverse: bool = False, magnitude: float = 1.0, out=None,
           stream=None):
    """Rotate x [T][heads][dims] bf16 by its tokens' positions [T] int32 (``mla_rotate``) -> out.

    x: last dim contiguous, otherwise strided (part of each head: ``q[..., 128:]``); out: the same shape, or x
    itself to rotate in place; otherwise it must not overlap x.  table: ``rope_table_scaled``'s, or ``rope_table``'s for 64
    dims.  layout "interleaved" turns the pairs (2i, 2i + 1), "half" the pairs (i, i + dims / 2).  inverse
    rotates back (the gradient of a rotation); magnitude multiplies the result.  A negative position
    leaves its token's rows of out as they were.
    """
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {tuple(_LAYOUTS)}, got {layout!r}")
    if stream is None:
        r = (B._host or B._native()).rotate(x, positions, table, _LAYOUTS[layout], bool(inverse), magnitude, out)
        if r is not None:
            return B._made(r, "mla_rotate")
    import torch
    index = _index_of(x, "x", 3, torch.bfloat16)
    T, heads, dims = x.shape
    if dims not in ROTARY_DIMS:
        raise ValueError(f"x's last dimension must be one of {ROTARY_DIMS}, got {dims}")
    src = _strided(x, "x", torch.bfloat16, (T, heads, dims), index)
    pos = _dense(positions, "positions", torch.int32, (T,), index, 4)
    tab = _dense(table, "table", torch.float32, (dims,), index, 4)
    with _launch_on(index, stream, x, positions, table, out):
        if out is None:
            out = torch.empty((T, heads, dims), dtype=torch.bfloat16, device=x.device)
        dst = _strided(out, "out", torch.bfloat16, (T, heads, dims), index)
        _check(load_library().mla_rotate(T, heads, dims, src[0], *src[1:], pos, tab, _LAYOUTS[layout], int(bool(inverse)),
                                         float(magnitude), dst[0], *dst[1:], _current_stream(index)), "mla_rotate")
    return out


# ----------------------------------------------------------------------------- residual and norm

def _rows(t, name, index, T, N):
    """Address and row stride of an input [T][N]."""
    import torch
    return _strided(t, name, torch.bfloat16, (T, N), index)


def residual_norm(x, residual, weight, *, rms_eps: float = DEFAULT_RMS_EPS, out=None, residual_out=None, stream=None):
    """Residual addition and RMSNorm (``mla_residual_norm``) -> (out [T][hidden] bf16, residual_out).

    z = x + residual, out = z / sqrt(mean z^2 + rms_eps) * weight, residual_out = z, each rounded once.
    x and residual [T][hidden] bf16 (rows strided at will; hidden a multiple of 8 up to 16384), weight
    [hidden] bf16.  residual None: x alone, and no residual_out (None).  residual_out may be residual itself.
    """
    r = None
    if stream is None:
        r = (B._host or B._native()).residual_norm(x, residual, weight, rms_eps, -1, out, None, residual_out)
        if r is not None:
            o, _, kept = B._made(r, "mla_residual_norm")
            return o, kept
    import torch
    index, T, N, args = _norm_args(x, residual, weight, residual_out)
    with _launch_on(index, stream, x, residual, weight, out, residual_out):
        out = _out(out, "out", torch.bfloat16, (T, N), index)
        if residual is not None:
            residual_out = _out(residual_out, "residual_out", torch.bfloat16, (T, N), index)
        _check(load_library().mla_residual_norm(T, N, *args, float(rms_eps), out.data_ptr(),
                                                None if residual is None else residual_out.data_ptr(),
                                                _current_stream(index)), "mla_residual_norm")
    return out, residual_out


def residual_norm_fp8(x, residual, weight, *, group: int = 128, rms_eps: float = DEFAULT_RMS_EPS, codes=None, scales=None,
                      residual_out=None, stream=None):
    """``residual_norm`` in 8 bits (``mla_residual_norm_fp8``) -> (codes, scales, residual_out).

    codes [T][hidden] float8_e4m3fn and scales [T][ceil(hidden / group)] fp32 (group 128, or 0: one scale per
    row, [T][1]): the norm is code * scale, with scale = max |norm| / 448 over the group's values.
    """
    if group not in (0, 128):
        raise ValueError(f"group must be 128 or 0, got {group}")
    if stream is None:
        r = (B._host or B._native()).residual_norm(x, residual, weight, rms_eps, group, codes, scales, residual_out)
        if r is not None:
            return B._made(r, "mla_residual_norm_fp8")
    import torch
    index, T, N, args = _norm_args(x, residual, weight, residual_out)
    with _launch_on(index, stream, x, residual, weight, codes, scales, residual_out):
        codes = _out(codes, "codes", torch.float8_e4m3fn, (T, N), index)
        scales = _out(scales, "scales", torch.float32, (T, -(-N // group) if group else 1), index)
        if residual is not None:
            residual_out = _out(residual_out, "residual_out", torch.bfloat16, (T, N), index)
        _check(load_library().mla_residual_norm_fp8(T, N, *args, float(rms_eps), group, codes.data_ptr(),
                                                    scales.data_ptr(),
                                                    None if residual is None else residual_out.data_ptr(),
                                                    _current_stream(index)), "mla_residual_norm_fp8")
    return codes, scales, residual_out


def _norm_args(x, residual, weight, residual_out):
    import torch
    index = _index_of(x, "x", 2, torch.bfloat16)
    T, N = x.shape
    if N % 8 or N > 16384:
        raise ValueError(f"x's rows must be a multiple of 8 values and at most 16384, got {N}")
    src = _rows(x, "x", index, T, N)
    res = (None, 8) if residual is None else _rows(residual, "residual", index, T, N)
    w = _dense(weight, "weight", torch.bfloat16, (N,), index)
    if residual is None and residual_out is not None:
        raise ValueError("residual_out without residual")
    return index, T, N, (*src, *res, w)


# ----------------------------------------------------------------------------- attention of chunks

CHUNK_SCRATCH_BYTES = 16 << 30


@dataclass
class ChunkPlan:
    """The tiles and pages of a step's chunks in a device workspace (one step's lengths and offsets)."""
    batch: int
    tokens: int
    max_pages: int
    kv_tokens: int
    workspace: object   # torch.uint8 CUDA tensor, owned by this ChunkPlan
    scratch: dict = field(default_factory=dict)   # heads and bytes of a call's own scratch, by whether the cache is fp8

    def problem(self) -> _Chunk:
        return _Chunk(self.batch, self.tokens, NUM_HEADS, PAGE_SIZE, self.max_pages, 0, self.kv_tokens)


def chunk_plan(seq_lens, token_offsets, *, tokens: int, max_pages_per_seq: int, kv_tokens: int | None = None,
               workspace=None, stream=None) -> ChunkPlan:
    """Lay out a step's chunks on the device (``mla_chunk_plan``).

    seq_lens [B] int32 (cached keys, the chunks included), token_offsets [B + 1] int32 (request b's tokens are
    rows token_offsets[b] .. token_offsets[b + 1] - 1 of the token arrays), tokens: rows of those arrays (may
    exceed token_offsets[B]: padding).  kv_tokens: at least the sum of the seq_lens, each rounded up to whole
    pages of 64 (by default what the table's width allows): it sizes the scratch of ``chunk_attend``, 64 KB a
    token, so a server passes what it knows.  The plan serves every layer of the step; calls that share it must be
    ordered, and it may be dropped once the last is enqueued.
    """
    import torch
    if not (0 < tokens < 1 << 31 and 0 < max_pages_per_seq < 1 << 31 and (kv_tokens is None or 0 < kv_tokens < 1 << 62)):
        _int(tokens, "tokens")               # (what the fields hold is refused by the C ABI)
        _int(max_pages_per_seq, "max_pages_per_seq")
        _int(kv_tokens or 0, "kv_tokens", 62)
    index = _index_of(seq_lens, "seq_lens", 1, torch.int32)
    n = seq_lens.shape[0]
    if kv_tokens is None:
        kv_tokens = n * int(max_pages_per_seq) * PAGE_SIZE
    kv_tokens = -(-int(kv_tokens) // PAGE_SIZE) * PAGE_SIZE
    if stream is None:
        r = (B._host or B._native()).chunk_plan(seq_lens, token_offsets, tokens, max_pages_per_seq, kv_tokens, workspace)
        if r is not None:
            return ChunkPlan(n, tokens, max_pages_per_seq, kv_tokens, B._made(r, "mla_chunk_plan"))
    sl = _dense(seq_lens, "seq_lens", torch.int32, (n,), index, 4)
    off = _dense(token_offsets, "token_offsets", torch.int32, (n + 1,), index, 4)
    p = ChunkPlan(n, int(tokens), int(max_pages_per_seq), kv_tokens, workspace)
    prob, lib = p.problem(), load_library()
    with _launch_on(index, stream, seq_lens, token_offsets, workspace):
        if workspace is None:
            size = ctypes.c_size_t(0)
            _check(lib.mla_chunk_workspace_size(ctypes.byref(prob), ctypes.byref(size)), "mla_chunk_workspace_size")
            p.workspace = torch.empty(size.value, dtype=torch.uint8, device=seq_lens.device)
        ws, nbytes = B._bytes(p.workspace, "workspace", index)
        p.workspace.record_stream(torch.cuda.current_stream())
        _check(lib.mla_chunk_plan(ctypes.byref(prob), sl, off, ws, nbytes, _current_stream(index)), "mla_chunk_plan")
    return p


def chunk_scratch_size(p: ChunkPlan, heads: int = NUM_HEADS, *, fp8: bool = False) -> int:
    """Bytes of the scratch that holds the keys and values of `heads` heads at once (``mla_chunk_scratch_size``)."""
    size, prob, heads = ctypes.c_size_t(0), p.problem(), _int(heads, "heads")
    with _launch_on(p.workspace.get_device(), None):
        _check(load_library().mla_chunk_scratch_size(ctypes.byref(prob), heads, int(bool(fp8)), ctypes.byref(size)),
               "mla_chunk_scratch_size")
    return size.value


def chunk_attend(p: ChunkPlan, q_nope, q_rope, w_uk, w_uv, kv_cache, block_table, *, scale: float = DEFAULT_SCALE,
                 out=None, lse=None, scratch=None, stream=None):
    """Attention of chunks of prompts over the paged cache (``mla_chunk_attend``) -> out [T][128][128] bf16.

    q_nope [T][128][128] and q_rope [T][128][64] bf16 (rotated; last dim contiguous, otherwise strided: both may
    be views of one projection's output), w_uk and w_uv [128][128][512] bf16, kv_cache [pages][64][576] with the
    chunks' own rows appended, block_table [B][max_pages] int32.  A token sees its request's slots up to its own.
    out is what ``epilog_oproj`` takes; rows behind the last request are not written.  lse: an optional fp32
    [T][128] to fill.  ``check(p)`` reads the status bits.

    Keys and values of all heads are worked out once per call from the cached rows, into scratch: a uint8 tensor of
    ``chunk_scratch_size(p, heads)`` bytes for as many heads at a time as it shall hold, by default one for
    the call with all 128, or as many as CHUNK_SCRATCH_BYTES hold.  A request of few tokens (some 100 at most) over a long
    context is computed in the absorbed form instead (``query``, the tree step's attention, ``epilog_uv``): the plan takes
    a form for each request, or for the step where its sizes say enough (``mla_chunk.h``).
    """
    return _attend(p, q_nope, q_rope, w_uk, w_uv, kv_cache, block_table, scale, out, lse, scratch, stream, False)


def chunk_attend_fp8(p: ChunkPlan, q_nope, q_rope, w_uk, w_uv, kv_cache_fp8, block_table, *, scale: float = DEFAULT_SCALE,
                     out=None, lse=None, scratch=None, stream=None):
    """``chunk_attend`` over an fp8 cache (``mla_chunk_attend_fp8``; uint8 [pages][64][656])."""
    return _attend(p, q_nope, q_rope, w_uk, w_uv, kv_cache_fp8, block_table, scale, out, lse, scratch, stream, True)


def _own_scratch(p, fp8, call):
    """call(bytes) with a scratch for all heads at once, or for as many as CHUNK_SCRATCH_BYTES and the memory hold."""
    import torch
    heads, need = p.scratch.get(fp8, (NUM_HEADS, None))
    if need is None:
        need = chunk_scratch_size(p, heads, fp8=fp8)
        while need > CHUNK_SCRATCH_BYTES and heads > 1 and chunk_scratch_size(p, heads // 2, fp8=fp8) < need:
            heads //= 2      # (the absorbed form's does not go by heads)
            need = chunk_scratch_size(p, heads, fp8=fp8)
        p.scratch[fp8] = heads, need
    while True:
        try:
            return call(need)
        except torch.OutOfMemoryError:
            less = chunk_scratch_size(p, heads // 2, fp8=fp8) if heads > 1 else need
            if less >= need:
                raise
            heads, need = p.scratch[fp8] = heads // 2, less


def _attend(p, q_nope, q_rope, w_uk, w_uv, kv_cache, block_table, scale, out, lse, scratch, stream, fp8):
    if scratch is not None and not hasattr(scratch, "data_ptr"):
        raise TypeError("scratch must be a torch.Tensor or None")
    if scratch is None:
        return _own_scratch(p, fp8, lambda need: _attend_in(p, q_nope, q_rope, w_uk, w_uv, kv_cache, block_table, scale, out,
                                                            lse, need, stream, fp8))
    return _attend_in(p, q_nope, q_rope, w_uk, w_uv, kv_cache, block_table, scale, out, lse, scratch, stream, fp8)


def _attend_in(p, q_nope, q_rope, w_uk, w_uv, kv_cache, block_table, scale, out, lse, scratch, stream, fp8):
    """One call with a scratch: a tensor, or how many bytes of it to make."""
    T, ws = p.tokens, p.workspace
    if stream is None:
        r = (B._host or B._native()).chunk_attend(p.batch, T, p.max_pages, p.kv_tokens, ws, q_nope, q_rope, w_uk, w_uv,
                                                  kv_cache, block_table, scale, out, lse, scratch, fp8)
        if r is not None:
            return B._made(r, "mla_chunk_attend_fp8" if fp8 else "mla_chunk_attend")
    import torch
    index = ws.get_device()
    q = (*_strided(q_nope, "q_nope", torch.bfloat16, (T, NUM_HEADS, D_NOPE), index),
         *_strided(q_rope, "q_rope", torch.bfloat16, (T, NUM_HEADS, D_ROPE), index))
    uk = _dense(w_uk, "w_uk", torch.bfloat16, (NUM_HEADS, D_NOPE, D_LATENT), index)
    uv = _dense(w_uv, "w_uv", torch.bfloat16, (NUM_HEADS, D_V, D_LATENT), index)
    cache = _cache_ptr(kv_cache, fp8, index)
    bt = _dense(block_table, "block_table", torch.int32, (p.batch, p.max_pages), index, 4)
    to_lse = None if lse is None else _dense(lse, "lse", torch.float32, (T, NUM_HEADS), index, 4)
    lib = load_library()
    with _launch_on(index, stream, ws, q_nope, q_rope, w_uk, w_uv, kv_cache, block_table, out, lse, scratch):
        out = _out(out, "out", torch.bfloat16, (T, NUM_HEADS, D_V), index)
        if isinstance(scratch, int):
            scratch = torch.empty(scratch, dtype=torch.uint8, device=ws.device)
        room = B._bytes(scratch, "scratch", index)
        ws.record_stream(torch.cuda.current_stream())
        prob = p.problem()
        f = lib.mla_chunk_attend_fp8 if fp8 else lib.mla_chunk_attend
        _check(f(ctypes.byref(prob), *q, uk, uv, cache, kv_cache.shape[0], bt, float(scale), out.data_ptr(), to_lse,
                 ws.data_ptr(), ws.numel(), *room, _current_stream(index)),
               "mla_chunk_attend_fp8" if fp8 else "mla_chunk_attend")
    return out
