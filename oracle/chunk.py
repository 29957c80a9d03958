"""64-bit oracle of a layer step over chunks of prompts (test infrastructure only).

Only the test suite and ``__graft_entry__.smoke()`` may import this module.  Plain torch in
float64 on whatever device the inputs are: rotary positions in either layout, scaled for long
contexts or not; residual addition and RMSNorm, in e4m3 codes with scales too; the attention of
a request's chunk over its cached rows, written out with every head's keys and values.

Pins: ``tests/test_chunk_pins.py``.
"""

from __future__ import annotations

import math

import torch

PAGE = 64
E4M3_MAX = 448.0


def rates(dims: int, base: float = 10000.0, factor: float = 1.0, original: int = 4096, fast: float = 32.0, slow: float = 1.0):
    """Radians per position of each pair: base^(-2i / dims), mixed with 1 / factor of it by how often the pair turns."""
    out = []
    ends = [dims * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (fast, slow)]
    low, high = max(0, math.floor(ends[0])), min(dims - 1, math.ceil(ends[1]))
    for i in range(dims // 2):
        r = base ** (-2 * i / dims)
        w = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
        out.append(r * (1 - w) + r / factor * w)
    return torch.tensor(out, dtype=torch.float64)


def rotate(x, positions, rate, *, half: bool = False, magnitude: float = 1.0, inverse: bool = False):
    """x [T][heads][dims] turned by positions [T] times rate [dims / 2]."""
    x = x.double()
    a = positions.to(x.device).double()[:, None] * rate.to(x.device)
    c, s = magnitude * a.cos()[:, None], magnitude * a.sin()[:, None] * (-1 if inverse else 1)
    out = torch.empty_like(x)
    n = x.shape[-1] // 2
    first, second = (slice(0, n), slice(n, 2 * n)) if half else (slice(0, None, 2), slice(1, None, 2))
    out[..., first] = x[..., first] * c - x[..., second] * s
    out[..., second] = x[..., first] * s + x[..., second] * c
    return out


def residual_norm(x, residual, weight, eps: float):
    """(y, z) of rows: z = x + residual, y = z / sqrt(mean z^2 + eps) * weight."""
    z = x.double() if residual is None else x.double() + residual.double()
    return z / (z.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double(), z


def group_scales(y, group: int):
    """[T][groups] of max |y| / 448 (1 for a group of zeros), and the same for every value."""
    T, N = y.shape
    g = group or N
    top = torch.stack([y[:, i:i + g].abs().amax(1) for i in range(0, N, g)], 1) / E4M3_MAX
    top = torch.where(top == 0, torch.ones_like(top), top)
    return top, top.repeat_interleave(g, 1)[:, :N]


def cache_rows(cache, table_row, length: int):
    """Rows [length][576] of one request from a bf16 cache or an fp8 one (uint8 rows of 656 bytes)."""
    pages = table_row[:-(-length // PAGE)].long().to(cache.device)
    r = cache[pages].reshape(-1, cache.shape[-1])[:length]
    if cache.dtype == torch.uint8:
        size = r[:, 640:644].contiguous().view(torch.float32).double()
        return torch.cat([r[:, :512].contiguous().view(torch.float8_e4m3fn).double(),
                          r[:, 512:640].contiguous().view(torch.bfloat16).double()], 1) * size
    return r.double()


def chunk_attend(q, w_uk, w_uv, cache, block_table, seq_lens, offsets, *, scale: float):
    """(o [T][H][128], lse [T][H], spread, reach) of ragged chunks; q [T][H][192] rotated; rows of no request are NaN.

    spread = sum_j w_j |v_j|, what a relative error of the weights is multiplied by; reach [T][H] = the largest
    scale * sum_d |q_d k_d| over the no-position dims of the keys seen, what the relative rounding of keys is
    multiplied by in a score.
    """
    T, H = q.shape[:2]
    nan = dict(fill_value=math.nan, dtype=torch.float64, device=q.device)
    o, lse, spread = torch.full((T, H, w_uv.shape[1]), **nan), torch.full((T, H), **nan), torch.full((T, H, w_uv.shape[1]), **nan)
    reach = torch.full((T, H), **nan)
    dn = w_uk.shape[1]
    for b in range(len(seq_lens)):
        t0, t1, L = int(offsets[b]), int(offsets[b + 1]), int(seq_lens[b])
        if t0 == t1:
            continue
        rows = cache_rows(cache, block_table[b], L)
        place = torch.arange(L - (t1 - t0), L, device=q.device)
        unseen = torch.arange(L, device=q.device)[None, :] > place[:, None]
        for h in range(H):
            k, v = rows[:, :512] @ w_uk[h].double().T, rows[:, :512] @ w_uv[h].double().T
            qh = q[t0:t1, h].double()
            x = scale * (qh @ torch.cat([k, rows[:, 512:]], 1).T)
            x = x.masked_fill(unseen, -math.inf)
            lse[t0:t1, h] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[t0:t1, h][:, None])
            p = torch.where(unseen, torch.zeros_like(p), p)
            clean = torch.where(unseen.all(0)[:, None], torch.zeros_like(v), v)
            o[t0:t1, h] = _seen(p, clean, unseen)
            spread[t0:t1, h] = _seen(p, clean.abs(), unseen)
            reach[t0:t1, h] = (scale * (qh[:, :dn].abs() @ k.abs().T)).masked_fill(unseen, 0).amax(1)
    return o, lse, spread, reach


def _seen(p, v, unseen):
    """p @ v in which an unseen key counts nothing whatever it holds."""
    bad = ~torch.isfinite(v).all(1)
    if not bool(bad.any()):
        return p @ v
    out = p @ torch.where(bad[:, None], torch.zeros_like(v), v)
    out[(bad[None, :] & ~unseen).any(1)] = math.nan
    return out
