"""The operators of a step over chunks of prompts, and what is measured of them.

A server prefills long prompts in chunks: a few hundred to a few thousand new tokens of each of a
few requests go through a layer together.  Beside the append of their rows to the paged latent cache
(which ``operators.py`` measures) such a layer needs

  rotate   rotary positions of the chunk's queries: interleaved or half layout, 64 of a head's 192
           values, angles scaled for long contexts
  chunk    attention of the chunk's tokens over their requests' paged caches, earlier chunks and the
           chunk itself, in the form with per-head keys and values (192 and 128 values a head)
  norm     the layer's boundary: residual addition and root-mean-square norm, to bf16 or to 8 bits
           with a scale per 128 values or per row, as the next projections take them

Shapes: 128 heads, 512 latent and 64 rotary values per cached row, 64-token pages, hidden size 7168,
as everywhere in this library.  Where ``own`` is false the operators run as elementary torch operations.
"""

import math
import random

import numpy as np
import torch

own = False

H, DL, DR, DN, DV, PAGE = 128, 512, 64, 128, 128, 64
ROW = DL + DR
ROW8 = 656                     # fp8 row: 512 e4m3 codes, 64 bf16 rotary values, one fp32 scale, padding
SCALE = 192.0 ** -0.5
BASE, EPS = 10000.0, 1e-6
ORIGINAL = 4096                # context length that a model was trained on, where its positions are scaled
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token: the latency of the rotation
        {"name": "rotate_1", "op": "rotate", "tokens": 1, "heads": 128, "dims": 64, "half": False, "factor": 1.0, "far": 8192},
        # a few requests' tokens, half layout
        {"name": "rotate_333", "op": "rotate", "tokens": 333, "heads": 128, "dims": 64, "half": True, "factor": 1.0, "far": 32768},
        # a full chunk of a long prompt: positions past the training length, scaled
        {"name": "rotate_4097", "op": "rotate", "tokens": 4097, "heads": 128, "dims": 64, "half": False, "factor": 40.0, "far": 163840},
        # the end of a short prompt: latency
        {"name": "chunk_77", "op": "chunk", "fp8": False, "batch": 1, "least": 77, "most": 77, "lo": 700, "hi": 700, "layout": 1},
        # ragged chunks of a few requests, one slot of the batch without tokens
        {"name": "chunk_ragged", "op": "chunk", "fp8": False, "batch": 5, "least": 65, "most": 900, "lo": 900, "hi": 8192, "layout": 2},
        # a whole prompt at once
        {"name": "chunk_prompt", "op": "chunk", "fp8": False, "batch": 1, "least": 4096, "most": 4096, "lo": 4096, "hi": 4096, "layout": 3},
        # the last chunk of a long prompt
        {"name": "chunk_long", "op": "chunk", "fp8": False, "batch": 1, "least": 2048, "most": 2048, "lo": 32768, "hi": 32768, "layout": 4},
        # the fp8 cache
        {"name": "chunk_fp8", "op": "chunk", "fp8": True, "batch": 3, "least": 129, "most": 700, "lo": 2048, "hi": 12288, "layout": 5},
        # one token of a decode step
        {"name": "norm_1", "op": "norm", "tokens": 1, "hidden": 7168, "fp8": False, "group": 128},
        # a decode step of a batch, a scale per row
        {"name": "norm_fp8_61", "op": "norm", "tokens": 61, "hidden": 7168, "fp8": True, "group": 0},
        # a chunk
        {"name": "norm_2049", "op": "norm", "tokens": 2049, "hidden": 7168, "fp8": False, "group": 128},
        # several chunks together, blocks of 128 values
        {"name": "norm_fp8_8191", "op": "norm", "tokens": 8191, "hidden": 7168, "fp8": True, "group": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "chunk", "chunk", "norm"])
    if op == "rotate":
        return {"op": op, "tokens": _log(rng, 1, 4097), "heads": rng.choice([1, 16, 128, rng.randint(2, 128)]), "dims": rng.choice([32, 64, 64, 128]),
                "half": rng.random() < 0.5, "factor": rng.choice([1.0, 4.0, 40.0]), "far": _log(rng, 64, 1 << 20)}
    if op == "norm":
        return {"op": op, "tokens": _log(rng, 1, 8191), "hidden": 8 * rng.randint(8, 896), "fp8": rng.random() < 0.6, "group": rng.choice([0, 128])}
    batch, most = _log(rng, 1, 8), _log(rng, 1, 2048)
    hi = max(most, min(_log(rng, most, 32768), 32768 // batch, (2048 * 24576) // (batch * most)))
    return {"op": op, "fp8": rng.random() < 0.5, "batch": batch, "least": rng.randint(1, most), "most": most,
            "lo": rng.randint(most, hi), "hi": hi, "layout": rng.randrange(1 << 30)}


def _sizes(case):
    """(counts, lengths) of a case's requests: tokens of this step, and cached tokens with them."""
    r = random.Random(case["layout"])
    B = case["batch"]
    counts = [r.randint(case["least"], case["most"]) for _ in range(B)]
    lengths = [max(c, _log(r, case["lo"], case["hi"])) for c in counts]
    if B >= 4 and case["least"] < case["most"]:
        counts[r.randrange(B)] = 0            # a slot of the batch without tokens
    return counts, lengths


def work(case):
    if case["op"] == "rotate":
        n = case["tokens"] * case["heads"] * case["dims"]
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 3 * n}
    if case["op"] == "norm":
        T, N = case["tokens"], case["hidden"]
        scales = 4 * (-(-N // case["group"]) if case["group"] else 1) if case["fp8"] else 0
        return {"bytes": T * (6 * N + (N + scales if case["fp8"] else 2 * N)) + 2 * N, "flops": 6 * T * N}
    counts, lengths = _sizes(case)
    row = ROW8 if case["fp8"] else 2 * ROW
    T = sum(counts)
    keys = sum(L for L, c in zip(lengths, counts) if c)
    flops = 0
    for L, c in zip(lengths, counts):
        pairs = c * (L - c) + c * (c + 1) // 2
        # keys and values of every head once, then 192 + 128 products a pair; or the absorbed form, if that is less
        flops += min(2 * H * (DN + DV) * DL * L + 2 * H * (DN + DR + DV) * pairs if c else 0,
                     2 * H * (DN + DV) * DL * c + 2 * H * (ROW + DL) * pairs)
    return {"bytes": keys * row + 4 * H * DN * DL + 2 * T * H * (DN + DR + DV), "flops": flops}


# ------------------------------------------------------------------------------ inputs

def _quantise(rows):
    """fp8 rows (bytes) of fp32 rows [..][576]."""
    c, k = rows[..., :DL], rows[..., DL:]
    top = c.abs().amax(-1, keepdim=True)
    s = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    out = torch.zeros(rows.shape[:-1] + (ROW8,), dtype=torch.uint8, device=rows.device)
    out[..., :DL] = (c / s).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    out[..., DL:DL + 2 * DR] = (k / s).to(torch.bfloat16).view(torch.uint8)
    out[..., DL + 2 * DR:DL + 2 * DR + 4] = s.contiguous().view(torch.uint8)
    return out


def _rows(cache):
    """fp32 rows [..][576] of a cache of either kind."""
    if cache.dtype != torch.uint8:
        return cache.float()
    c, k = cache[..., :DL].view(torch.float8_e4m3fn), cache[..., DL:DL + 2 * DR].view(torch.bfloat16)
    return torch.cat([c.float(), k.float()], -1) * cache[..., DL + 2 * DR:DL + 2 * DR + 4].view(torch.float32)


def _rates(dims, factor, device):
    """Radians per position of each pair, in 64 bits; scaled for long contexts (YaRN) if factor is over 1:
    pairs that turn often within the original length keep their rate, slow ones are slowed by the factor."""
    i = torch.arange(dims // 2, dtype=torch.float64, device=device)
    rate = torch.tensor(BASE, dtype=torch.float64, device=device) ** (i * (-2.0 / dims))
    if factor <= 1:
        return rate

    def pair_of(turns):
        return dims * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(BASE))

    low, high = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), dims - 1)
    slow = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return rate / factor * slow + rate * (1 - slow)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(int(seed))
    gd = torch.Generator(device=dev).manual_seed(int(seed) + 1)
    bf = torch.bfloat16

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gd, device=dev) * std).to(bf)

    s = {"op": case["op"]}
    if case["op"] == "rotate":
        T, dims = case["tokens"], case["dims"]
        s["x"] = normal(T, case["heads"], DN + dims)[..., DN:]      # the last part of each head
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, dtype=torch.int32).to(dev)
        s["half"] = case["half"]
        s["magnitude"] = 0.1 * math.log(case["factor"]) + 1.0
        s["rate"] = _rates(dims, case["factor"], dev)
        # the model's rotary table: turns per position as a sum of two floats
        turns = s["rate"] / (2 * math.pi)
        hi = turns.float()
        s["table"] = torch.cat([hi, (turns - hi.double()).float()])
        return s
    if case["op"] == "norm":
        T, N = case["tokens"], case["hidden"]
        s["x"], s["residual"] = normal(T, N, std=0.5), normal(T, N, std=2.0)
        s["weight"] = (1 + 0.1 * torch.randn(N, generator=gd, device=dev)).to(bf)
        s["fp8"], s["group"] = case["fp8"], case["group"]
        return s
    counts, lengths = _sizes(case)
    T = sum(counts)
    s["q"] = normal(T, H, DN + DR)                       # one projection's output, its rotary part rotated
    s["w_uk"], s["w_uv"] = normal(H, DN, DL, std=DL ** -0.5), normal(H, DV, DL, std=DL ** -0.5)
    s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=dev)
    s["seq_lens"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    s["most"] = max(counts)
    pages = [-(-L // PAGE) for L in lengths]
    total, width = sum(pages), max(pages)
    s["kv_tokens"] = total * PAGE                        # a server knows how many pages its requests hold
    order = torch.randperm(total, generator=g).numpy()
    table = np.full((len(counts), width), -1, np.int32)
    for b, n in enumerate(pages):
        table[b, :n] = order[sum(pages[:b]):sum(pages[:b]) + n]
    s["block_table"] = torch.from_numpy(table).to(dev)
    cache = torch.randn(total, PAGE, ROW, generator=gd, device=dev)
    s["cache"] = _quantise(cache) if case["fp8"] else cache.to(bf)
    return s


# ------------------------------------------------------------------------------ the plain forms

def _plain_rotate(s):
    a = s["positions"].double()[:, None] * s["rate"]
    c, n = ((f * s["magnitude"]).float()[:, None] for f in (a.cos(), a.sin()))
    x = s["x"].float()
    if s["half"]:
        u, v = x.chunk(2, -1)
        return torch.cat([u * c - v * n, u * n + v * c], -1).to(torch.bfloat16)
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * c - v * n, u * n + v * c], -1).flatten(-2).to(torch.bfloat16)


def _plain_norm(s):
    z = s["x"].float() + s["residual"].float()
    y = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    kept = z.to(torch.bfloat16)
    if not s["fp8"]:
        return y.to(torch.bfloat16), kept
    T, N = y.shape
    group = s["group"] or N
    blocks = torch.nn.functional.pad(y, (0, -N % group)).view(T, -1, group)
    top = blocks.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    codes = (blocks / scale).clamp(-E4M3_MAX, E4M3_MAX).view(T, -1)[:, :N].to(torch.float8_e4m3fn)
    return codes, scale[..., 0], kept


def _plain_chunk(s):
    T, B, N = s["q"].shape[0], s["seq_lens"].shape[0], s["most"]
    off = s["offsets"].long()
    counts = off[1:] - off[:-1]
    n = torch.arange(N, device=off.device)
    pick = (off[:-1, None] + n).clamp(max=T - 1)                                   # [B][N]
    q = s["q"].float()[pick].transpose(1, 2) * SCALE                               # [B][H][N][192]
    kv = _rows(s["cache"][s["block_table"].long().clamp(min=0)]).view(B, 1, -1, ROW)
    c, k_rope = kv[..., :DL], kv[..., DL:]
    k = torch.matmul(c, s["w_uk"].float().transpose(1, 2))                         # [B][H][keys][128]
    x = torch.matmul(q, torch.cat([k, k_rope.expand(-1, H, -1, -1)], -1).transpose(2, 3))
    place = (s["seq_lens"].long() - counts)[:, None] + n                           # [B][N] slots of the tokens
    hidden = torch.arange(kv.shape[2], device=off.device) > place[..., None]
    x.masked_fill_(hidden[:, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, torch.matmul(c, s["w_uv"].float().transpose(1, 2))) / total
    t = torch.arange(T, device=off.device)
    b = torch.searchsorted(off[1:], t, right=True)
    return o[b, :, t - off[b]].to(torch.bfloat16)


# ------------------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if not own:
        return {"rotate": _plain_rotate, "norm": _plain_norm, "chunk": _plain_chunk}[op](s)
    import mla_decode_attention_02_gb300 as mla
    if op == "rotate":
        return mla.rotate(s["x"], s["positions"], table=s["table"], layout="half" if s["half"] else "interleaved",
                          magnitude=s["magnitude"])
    if op == "norm":
        if s["fp8"]:
            return mla.residual_norm_fp8(s["x"], s["residual"], s["weight"], group=s["group"], rms_eps=EPS)
        return mla.residual_norm(s["x"], s["residual"], s["weight"], rms_eps=EPS)
    p = mla.chunk_plan(s["seq_lens"], s["offsets"], tokens=s["q"].shape[0], max_pages_per_seq=s["block_table"].shape[1],
                       kv_tokens=s["kv_tokens"])
    attend = mla.chunk_attend_fp8 if s["cache"].dtype == torch.uint8 else mla.chunk_attend
    return attend(p, s["q"][..., :DN], s["q"][..., DN:], s["w_uk"], s["w_uv"], s["cache"], s["block_table"], scale=SCALE)


# ------------------------------------------------------------------------------ in 64 bits

def _e4m3_64(x):
    """The e4m3 values nearest to x (ties to even, saturating), in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_rotate(case, s):
    d = case["dims"]
    i = np.arange(d // 2)
    rate = np.exp(i * (-2.0 * math.log(BASE) / d))
    if case["factor"] > 1:
        edge = [d / 2 * math.log(ORIGINAL / (2 * math.pi * turns), BASE) for turns in (32, 1)]
        low, high = max(0, math.floor(edge[0])), min(d - 1, math.ceil(edge[1]))
        keep = 1 - np.clip((i - low) / max(high - low, 1e-3), 0, 1)
        rate = rate * (keep + (1 - keep) / case["factor"])
    x = s["x"].double()
    pairs = x.unflatten(-1, (2, d // 2)).transpose(-1, -2) if case["half"] else x.unflatten(-1, (d // 2, 2))
    angle = s["positions"].double()[:, None] * torch.from_numpy(rate).cuda()
    turn = torch.polar(torch.full_like(angle, 1 + math.log(case["factor"]) / 10), angle)[:, None]
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    return (y.transpose(-1, -2) if case["half"] else y).flatten(-2)


def _exact_norm(case, s):
    z = s["x"].double() + s["residual"].double()
    T, N = z.shape
    size = torch.linalg.vector_norm(z, dim=1, keepdim=True)
    y = z / torch.sqrt(size * size / N + EPS) * s["weight"].double()
    if not case["fp8"]:
        return y, z
    codes, scales = torch.empty_like(y), []
    step = case["group"] or N
    for at in range(0, N, step):
        part = y[:, at:at + step]
        scales.append(part.abs().amax(1) / E4M3_MAX)
        codes[:, at:at + step] = _e4m3_64(part / scales[-1][:, None])
    return codes, torch.stack(scales, 1), z


def _exact_chunk(case, s):
    counts, lengths = _sizes(case)
    out, t = [], 0
    for b, (c, L) in enumerate(zip(counts, lengths)):
        if not c:
            continue
        keys = s["cache"][s["block_table"][b, :-(-L // PAGE)].long()].reshape(-1, s["cache"].shape[-1])[:L]
        if case["fp8"]:
            code, rope, size = keys[:, :DL].view(torch.float8_e4m3fn), keys[:, DL:DL + 2 * DR].view(torch.bfloat16), keys[:, DL + 2 * DR:DL + 2 * DR + 4].view(torch.float32)
            keys = torch.cat([code.double(), rope.double()], 1) * size.double()
        keys = keys.double()
        seen = torch.ones(c, L, dtype=torch.bool, device="cuda").tril(L - c)
        heads = []
        for h in range(H):
            key = torch.cat([keys[:, :DL] @ s["w_uk"][h].double().T, keys[:, DL:]], 1)
            x = torch.where(seen, s["q"][t:t + c, h].double() @ key.T * SCALE, -math.inf)
            heads.append(torch.softmax(x, 1) @ (keys[:, :DL] @ s["w_uv"][h].double().T))
        out.append(torch.stack(heads, 1))
        t += c
    return torch.cat(out)


def exact(case, seed):
    return {"rotate": _exact_rotate, "norm": _exact_norm, "chunk": _exact_chunk}[case["op"]](case, prepare(case, seed))
