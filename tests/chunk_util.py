"""Inputs of the chunk tests: ragged chunks over a paged pool, drawn from a seed (no attention arithmetic)."""

import numpy as np
import torch

PAGE = 64


def case(counts, lens, seed=0, pad=0, spare=2, width=0, device="cuda", fp8=False, poison=True, hold=None):
    """Chunks of counts[b] tokens at the end of lens[b] cached ones.

    With poison every slot past a request's end and every spare page holds NaN, and table entries past the end are
    outside the pool.  hold: {(b, slot): value}, rows to fill with a value.
    """
    g = torch.Generator(device=device).manual_seed(seed)
    rng = np.random.default_rng(seed)
    bf = torch.bfloat16
    need = [-(-L // PAGE) if n else 0 for n, L in zip(counts, lens)]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(counts), max(max(need), 1, width)), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    T = sum(counts) + pad

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=device) * std).to(bf)

    cache = normal(pages, PAGE, 576)
    if poison:
        used = np.zeros(pages, bool)
        for b, (n, L) in enumerate(zip(counts, lens)):
            if n:
                used[table[b, :need[b]]] = True
                if L % PAGE:
                    cache[int(table[b, L // PAGE]), L % PAGE:] = float("nan")
        cache[torch.from_numpy(~used).to(device)] = float("nan")
    for (b, slot), value in (hold or {}).items():
        cache[int(table[b, slot // PAGE]), slot % PAGE] = value
    c = {"counts": list(counts), "T": T, "n": sum(counts), "kv_tokens": sum(need) * PAGE,
         "seq_lens": torch.tensor(lens, dtype=torch.int32, device=device),
         "offsets": torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=device),
         "block_table": torch.from_numpy(table).to(device), "q": normal(T, 128, 192),
         "w_uk": normal(128, 128, 512, std=512 ** -0.5), "w_uv": normal(128, 128, 512, std=512 ** -0.5), "cache": cache}
    if fp8:
        c["cache"] = quantise(cache)
    return c


def quantise(cache):
    """fp8 rows (uint8, 656 bytes) of bf16 ones; a row that holds NaN becomes NaN codes and a NaN scale."""
    x = cache.float()
    c, k = x[..., :512], x[..., 512:]
    top = c.abs().amax(-1, keepdim=True)
    s = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    out = torch.zeros(x.shape[:-1] + (656,), dtype=torch.uint8, device=x.device)
    out[..., :512] = (c / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    out[..., 512:640] = (k / s).to(torch.bfloat16).view(torch.uint8)
    out[..., 640:644] = s.contiguous().view(torch.uint8)
    out[~torch.isfinite(x).all(-1)] = 0x7F
    return out
