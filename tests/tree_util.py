"""Inputs of the tree tests: ragged trees over a paged pool, drawn from a seed (no attention arithmetic)."""

import numpy as np
import torch

PAGE = 64


def masks_of(kind, n, rng):
    """Masks of one tree of n nodes: "chain", "tree" (ancestors and itself), "self", "bits" (anything), "none", "all"."""
    out = []
    for i in range(n):
        if kind == "chain":
            m = (1 << (i + 1)) - 1
        elif kind == "tree":
            m = (out[int(rng.integers(0, i))] if i else 0) | 1 << i
        elif kind == "self":
            m = 1 << i
        elif kind == "bits":
            m = int(rng.integers(0, 1 << 63)) | (int(rng.integers(0, 2)) << 63)
        elif kind == "all":
            m = (1 << 64) - 1
        else:
            m = 0
        out.append(m)
    return out


def case(counts, lens, kind="tree", seed=0, pad=0, spare=3, width=0):
    """Offsets, masks, lengths, block table (physical pages shuffled, unused entries out of the pool)."""
    rng = np.random.default_rng(seed)
    kinds = kind if isinstance(kind, (list, tuple)) else [kind] * len(counts)
    masks = [m & (1 << 64) - 1 for k, n in zip(kinds, counts) for m in masks_of(k, n, rng)] + [(1 << 64) - 1] * pad
    need = [(L + PAGE - 1) // PAGE if n else 0 for n, L in zip(counts, lens)]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(counts), max(max(need), 1, width)), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return {"counts": list(counts), "seq_lens": np.array(lens, np.int32), "pages": pages,
            "offsets": np.concatenate([[0], np.cumsum(counts)]).astype(np.int32),
            "masks": np.array(masks, np.uint64), "block_table": table, "T": sum(counts) + pad, "used": at, "order": order}


def tensors(c, seed=0, poison=True, quiet=False):
    """q and a bf16 cache for a case; with poison every slot past a request's end, every spare page, and
    every tree slot that none of its tree's masks names hold NaN.  quiet: zeros in their place."""
    g = torch.Generator().manual_seed(seed)
    bf = torch.bfloat16
    q_latent = torch.randn(c["T"], 128, 512, generator=g).to(bf)
    q_rope = torch.randn(c["T"], 128, 64, generator=g).to(bf)
    cache = torch.randn(c["pages"], PAGE, 576, generator=g).to(bf)
    if poison:
        fill = 0.0 if quiet else float("nan")
        spare = np.ones(c["pages"], bool)
        for b, n in enumerate(c["counts"]):
            L = int(c["seq_lens"][b])
            if n == 0:
                continue
            row = c["block_table"][b]
            spare[row[:(L + PAGE - 1) // PAGE]] = False
            if L % PAGE:
                cache[int(row[L // PAGE]), L % PAGE:] = fill
            seen = 0
            for t in range(c["offsets"][b], c["offsets"][b + 1]):
                seen |= int(c["masks"][t])
            for j in range(n):
                if not seen >> j & 1:
                    slot = L - n + j
                    cache[int(row[slot // PAGE]), slot % PAGE] = fill
        cache[torch.from_numpy(spare)] = fill
    return q_latent, q_rope, cache


def index_tensors(c, device="cuda"):
    return {"seq_lens": torch.from_numpy(c["seq_lens"]).to(device), "offsets": torch.from_numpy(c["offsets"]).to(device),
            "masks": torch.from_numpy(c["masks"].astype(np.int64)).to(device),
            "block_table": torch.from_numpy(c["block_table"]).to(device)}
