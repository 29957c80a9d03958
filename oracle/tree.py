"""fp64 oracle of a speculative step over trees of drafted tokens (test infrastructure only).

Only the test suite may import this module.  Plain numpy, one request at a time:
the cache rows of ragged tokens (RMSNorm, RoPE; the e4m3 row for an fp8 cache), the
attention of every node over its request's context and the nodes its mask names, and
the move of an accepted path's rows.  RoPE and RMSNorm are those of ``oracle.prolog``.

Pins: ``tests/test_tree_pins.py``.
"""

from __future__ import annotations

import numpy as np

from .prolog import _f64, rms_norm, rope

PAGE = 64


def visible(seq_len: int, nodes: int, mask: int) -> np.ndarray:
    """Which of the request's seq_len keys a node sees: the context, and the tree slots of its mask's bits."""
    seen = np.ones(seq_len, dtype=bool)
    for j in range(nodes):
        seen[seq_len - nodes + j] = bool(int(mask) >> j & 1)
    return seen


def keys(cache, table_row, seq_len: int) -> np.ndarray:
    """Rows [seq_len][576] of one request, fp64."""
    pages = np.asarray(table_row)[:(seq_len + PAGE - 1) // PAGE]
    return np.concatenate([_f64(cache[int(p)]) for p in pages], axis=0)[:seq_len] if seq_len else np.zeros((0, 576))


def tree_decode(q_latent, q_rope, cache, block_table, seq_lens, offsets, masks, *, scale: float):
    """(o [T][H][512], lse [T][H], spread [T][H][512]) in fp64; rows of no request are NaN.

    spread = sum_j w_j |v_j|: what a relative error of the weights is multiplied by.
    """
    ql, qr = _f64(q_latent), _f64(q_rope)
    T, H, DL = ql.shape
    o, lse, spread = np.full((T, H, DL), np.nan), np.full((T, H), np.nan), np.full((T, H, DL), np.nan)
    for b in range(len(seq_lens)):
        o0, n, L = int(offsets[b]), int(offsets[b + 1] - offsets[b]), int(seq_lens[b])
        if n == 0:
            continue
        rows = keys(cache, block_table[b], L)
        for i in range(n):
            t = o0 + i
            r = rows[visible(L, n, masks[t])]
            if len(r) == 0:
                o[t], lse[t], spread[t] = 0.0, -np.inf, 0.0
                continue
            x = scale * (ql[t] @ r[:, :DL].T + qr[t] @ r[:, DL:].T)
            m = x.max(axis=1, keepdims=True)
            w = np.exp(x - m)
            s = w.sum(axis=1, keepdims=True)
            o[t] = w @ r[:, :DL] / s
            spread[t] = w @ np.abs(r[:, :DL]) / s
            lse[t] = (m + np.log(s))[:, 0]
    return o, lse, spread


def token_slots(block_table, seq_lens, offsets):
    """(token, flat cache row, slot) of every token of every request."""
    out = []
    for b in range(len(seq_lens)):
        o0, o1 = int(offsets[b]), int(offsets[b + 1])
        for t in range(o0, o1):
            slot = int(seq_lens[b]) - o1 + t
            out.append((t, int(block_table[b][slot // PAGE]) * PAGE + slot % PAGE, slot))
    return out


def token_rows(kv_latent, k_pe, gamma, positions, *, rope_base: float = 10000.0, rms_eps: float = 1e-6):
    """(normalised latents [T][512], rotated k_pe [T][64]) in fp64."""
    return rms_norm(kv_latent, gamma, rms_eps), rope(k_pe, np.asarray(positions, np.int64), rope_base)


def commit(cache_rows, block_table, seq_lens, offsets, paths, path_lens):
    """(rows after the move, new lengths) of flat cache rows [pages * 64][..]: read all, then write."""
    out = np.array(cache_rows, copy=True)
    new = []
    for b in range(len(seq_lens)):
        n, L, k = int(offsets[b + 1] - offsets[b]), int(seq_lens[b]), int(path_lens[b])
        if n == 0:
            new.append(L)
            continue
        at = lambda i: int(block_table[b][(L - n + i) // PAGE]) * PAGE + (L - n + i) % PAGE  # noqa: E731
        for i in range(k):
            out[at(i)] = cache_rows[at(int(paths[b][i]))]
        new.append(L - n + k)
    return out, np.array(new, np.int32)
