"""The operators of a decode step over trees of drafted tokens, and what is measured of them.

A speculative decoding step of an MLA layer scores a small tree of drafted tokens per request
against the request's paged latent cache.  Four operators make that step:

  query    absorbed and rotated queries of T tokens at explicit positions
  append   RMSNorm, rotation and append of the tokens' rows to the paged cache (bf16 or fp8 rows)
  tree     attention of every tree node over its request's cache and its own ancestors
  commit   the rows of the accepted path move together, in every layer's cache

Shapes: 128 heads, 512 latent and 64 rotary values per cached row, 64-token pages, as everywhere
in this library.  Where ``own`` is false the operators run as elementary torch operations.
"""

import math
import random

import numpy as np
import torch

own = False

H, DL, DR, DN, PAGE = 128, 512, 64, 128, 64
ROW = DL + DR
ROW8 = 656                     # fp8 row: 512 e4m3 codes, 64 bf16 rotary values, one fp32 scale, padding
SCALE = 192.0 ** -0.5
BASE, EPS = 10000.0, 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one stream, one token: the latency of the query projection
        {"name": "query_1", "op": "query", "tokens": 1, "far": 8192},
        # a batch of ragged trees, an odd number of nodes
        {"name": "query_1537", "op": "query", "tokens": 1537, "far": 131072},
        # one stream's tree of 8 nodes
        {"name": "append_8", "op": "append", "fp8": False, "batch": 1, "least": 8, "most": 8, "lo": 700, "hi": 700, "layout": 1},
        # a prefill chunk of a few prompts, ragged
        {"name": "append_chunk", "op": "append", "fp8": False, "batch": 6, "least": 1, "most": 4096, "lo": 4097, "hi": 32768, "layout": 2},
        # a batch of trees into an fp8 cache
        {"name": "append_fp8", "op": "append", "fp8": True, "batch": 61, "least": 9, "most": 33, "lo": 64, "hi": 16384, "layout": 3},
        # one stream, one small tree, a short context: latency
        {"name": "tree_one", "op": "tree", "fp8": False, "batch": 1, "least": 8, "most": 8, "lo": 700, "hi": 700, "layout": 4},
        # an ordinary batch: ragged trees, mixed contexts, one slot of the batch without a request
        {"name": "tree_mixed", "op": "tree", "fp8": False, "batch": 13, "least": 5, "most": 16, "lo": 512, "hi": 8192, "layout": 5},
        # a full batch of 4096-token contexts with trees of 16 nodes
        {"name": "tree_uniform", "op": "tree", "fp8": False, "batch": 64, "least": 16, "most": 16, "lo": 4096, "hi": 4096, "layout": 6},
        # long contexts
        {"name": "tree_long", "op": "tree", "fp8": False, "batch": 2, "least": 12, "most": 12, "lo": 131072, "hi": 131072, "layout": 7},
        # the fp8 cache, large trees
        {"name": "tree_fp8", "op": "tree", "fp8": True, "batch": 17, "least": 12, "most": 41, "lo": 256, "hi": 8192, "layout": 8},
        # one layer group's caches, a small batch
        {"name": "commit_16", "op": "commit", "fp8": False, "batch": 3, "least": 7, "most": 16, "lo": 100, "hi": 8192, "layers": 4, "accept": 4, "layout": 9},
        # every layer's fp8 cache of a full batch
        {"name": "commit_fp8", "op": "commit", "fp8": True, "batch": 64, "least": 16, "most": 64, "lo": 64, "hi": 32768, "layers": 61, "accept": 6, "layout": 10},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["query", "append", "tree", "tree", "commit"])
    layout = rng.randrange(1 << 30)
    if op == "query":
        return {"op": op, "tokens": _log(rng, 1, 1537), "far": _log(rng, 64, 1 << 20)}
    fp8 = rng.random() < 0.5
    if op == "append":
        batch = _log(rng, 1, 64)
        most = _log(rng, 1, 64) if rng.random() < 0.5 else _log(rng, 64, 4096)
        most = max(1, min(most, 16384 // batch))
        lo = _log(rng, most, 32768)
        return {"op": op, "fp8": fp8, "batch": batch, "least": rng.randint(1, most), "most": most, "lo": lo, "hi": _log(rng, lo, 65536), "layout": layout}
    batch, most = _log(rng, 1, 64), _log(rng, 1, 64)
    if op == "tree":
        hi = _log(rng, most, min(131072, max(most, (64 * 16 * 4096) // (2 * batch * most))))
        return {"op": op, "fp8": fp8, "batch": batch, "least": rng.randint(1, most), "most": most, "lo": rng.randint(most, hi), "hi": hi, "layout": layout}
    lo = _log(rng, most, 32768)
    return {"op": op, "fp8": fp8, "batch": batch, "least": rng.randint(1, most), "most": most, "lo": lo, "hi": _log(rng, lo, 32768),
            "layers": _log(rng, 1, 61), "accept": rng.randint(1, 8), "layout": layout}


def _sizes(case):
    """(counts, lengths) of a case's requests: tokens of this step, and cached tokens with them."""
    r = random.Random(case["layout"])
    B = case["batch"]
    counts = [r.randint(case["least"], case["most"]) for _ in range(B)]
    lengths = [max(c, _log(r, case["lo"], case["hi"])) for c in counts]
    if B >= 8 and case["op"] == "tree" and case["least"] < case["most"]:
        counts[r.randrange(B)] = 0            # a slot of the batch without a request
    return counts, lengths


def work(case):
    if case["op"] == "query":
        T = case["tokens"]
        return {"bytes": 2 * T * H * (DN + DR + DL + DR) + 2 * H * DN * DL + 4 * T, "flops": 2 * T * H * DN * DL}
    counts, lengths = _sizes(case)
    row = ROW8 if case["fp8"] else 2 * ROW
    T = sum(counts)
    if case["op"] == "append":
        return {"bytes": T * (2 * ROW + row + 4), "flops": T * (4 * DL + 3 * DR)}
    if case["op"] == "commit":
        moved = sum(min(case["accept"], c) - 1 for c in counts)
        return {"bytes": max(1, moved) * case["layers"] * row * 2, "flops": 0}
    keys = sum(L for L, c in zip(lengths, counts) if c)
    pairs = sum(c * (L - c + 1) for L, c in zip(lengths, counts))   # a node sees the context and itself at least
    return {"bytes": keys * row + T * H * (2 * ROW + 2 * DL + 4), "flops": 2 * H * (ROW + DL) * pairs}


# ------------------------------------------------------------------------------ inputs

def _tree(r, n):
    """Parents of a tree of n nodes, each after its parent (node 0 is the root)."""
    return [-1] + [r.randint(max(0, i - 6), i - 1) for i in range(1, n)]


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


def _held(cache):
    """What an fp8 cache holds, as the values it stands for: codes, k_rope / s and s."""
    return (cache[..., :DL].view(torch.float8_e4m3fn), cache[..., DL:DL + 2 * DR].view(torch.bfloat16),
            cache[..., DL + 2 * DR:DL + 2 * DR + 4].view(torch.float32))


def _rows(cache):
    """fp32 rows [..][576] of a cache of either kind."""
    if cache.dtype != torch.uint8:
        return cache.float()
    c, k, s = _held(cache)
    return torch.cat([c.float(), k.float()], -1) * s


def _tokens_table(g, counts, lengths, whole):
    """(block_table, pages): the pages a step touches are a request's own; the others are its own too
    where the whole context is read, else any page."""
    B, width = len(counts), max((L + PAGE - 1) // PAGE for L in lengths)
    table = np.full((B, width), -1, np.int32)
    used = 0
    for b, (c, L) in enumerate(zip(counts, lengths)):
        n, first = (L + PAGE - 1) // PAGE, 0 if whole else (L - c) // PAGE
        if whole and c == 0:
            continue
        table[b, first:n] = np.arange(used, used + n - first)
        used += n - first
    order = torch.randperm(max(used, 1), generator=g).numpy()
    table = np.where(table >= 0, order[np.maximum(table, 0)], table)
    if not whole:
        for b, L in enumerate(lengths):
            n = (L + PAGE - 1) // PAGE
            gap = table[b, :n] < 0
            table[b, :n][gap] = np.arange(gap.sum()) % used
    return torch.from_numpy(table.astype(np.int32)), max(used, 1)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(int(seed))
    gd = torch.Generator(device=dev).manual_seed(int(seed) + 1)
    bf = torch.bfloat16

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gd, device=dev) * std).to(bf)

    s = {"op": case["op"], "status": torch.zeros(1, dtype=torch.int32, device=dev)}
    rate = torch.arange(DR // 2, dtype=torch.float64, device=dev) * (-2.0 / DR)
    s["rate"] = torch.tensor(BASE, dtype=torch.float64, device=dev) ** rate       # radians per position of each pair
    # the model's rotary table: turns per position as a sum of two floats
    turns = s["rate"] / (2 * math.pi)
    hi = turns.float()
    s["table"] = torch.cat([hi, (turns - hi.double()).float()])
    if case["op"] == "query":
        T = case["tokens"]
        s["q"] = normal(T, H, DN + DR)                   # one projection's output: both parts are views of it
        s["w_uk"] = normal(H, DN, DL, std=DN ** -0.5)
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, dtype=torch.int32).to(dev)
        return s
    counts, lengths = _sizes(case)
    r = random.Random(int(seed))
    T = sum(counts)
    s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=dev)
    s["seq_lens"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    s["most"] = max(counts)
    table, pages = _tokens_table(g, counts, lengths, case["op"] == "tree")
    s["block_table"] = table.to(dev)
    masks, depths = [], []
    for c in counts:
        up, m, d = _tree(r, c)[:c], [], []
        for i, p in enumerate(up):
            m.append((m[p] if p >= 0 else 0) | 1 << i)
            d.append(d[p] + 1 if p >= 0 else 0)
        masks += m if c <= 64 else []
        depths += d
    if case["op"] == "append":
        s["kv"] = normal(T, ROW)                         # the projection's output: latent and rotary part are views
        s["gamma"] = (1 + 0.1 * torch.randn(DL, generator=gd, device=dev)).to(bf)
        s["cache"] = torch.zeros((pages, PAGE, ROW8), dtype=torch.uint8, device=dev) if case["fp8"] else \
            torch.zeros((pages, PAGE, ROW), dtype=bf, device=dev)
        if case["most"] <= 64:                           # a tree's tokens stand at their depths, a chunk's at their slots
            first = np.repeat(np.array(lengths) - np.array(counts), counts)
            s["positions"] = torch.tensor(first + np.array(depths), dtype=torch.int32, device=dev)
        else:
            s["positions"] = None
        return s
    if case["op"] == "tree":
        s["q_latent"], s["q_rope"] = normal(T, H, DL), normal(T, H, DR)
        s["masks"] = torch.tensor(np.array(masks, dtype=np.uint64).astype(np.int64), device=dev)
        if case["fp8"]:
            s["cache"] = torch.empty((pages, PAGE, ROW8), dtype=torch.uint8, device=dev)
            for at in range(0, pages, 4096):
                n = min(4096, pages - at)
                s["cache"][at:at + n] = _quantise(torch.randn(n, PAGE, ROW, generator=gd, device=dev))
        else:
            s["cache"] = torch.empty((pages, PAGE, ROW), dtype=bf, device=dev)
            for at in range(0, pages, 4096):
                n = min(4096, pages - at)
                s["cache"][at:at + n] = normal(n, PAGE, ROW)
        return s
    # commit: node 0 and then deeper nodes; none of them lies in a slot that the pass overwrites with another's
    # row, so that a second pass finds the same rows
    paths = np.zeros((len(counts), max(min(case["accept"], c) for c in counts)), np.int32)
    took = []
    for b, c in enumerate(counts):
        n = min(case["accept"], c)
        k = r.randint(0, n) if c - n >= n else n         # nodes that stay where they are
        paths[b, :n] = list(range(k)) + sorted(r.sample(range(n, c), n - k))
        took.append(n)
    s["paths"] = torch.from_numpy(paths).to(dev)
    s["path_lens"] = torch.tensor(took, dtype=torch.int32, device=dev)
    if case["fp8"]:
        s["cache"] = torch.stack([_quantise(torch.randn(pages, PAGE, ROW, generator=gd, device=dev)) for _ in range(case["layers"])])
    else:
        s["cache"] = normal(case["layers"], pages, PAGE, ROW)
    return s


# ------------------------------------------------------------------------------ the plain forms

def _turn(x, positions, rate):
    """Rotates the pairs (2i, 2i + 1) of x [T][..][64] by position times rate, angles in 64 bits."""
    a = positions.double()[:, None] * rate
    c, s = a.cos().float(), a.sin().float()
    while c.dim() < x.dim():
        c, s = c[:, None], s[:, None]
    x = x.float()
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * c - v * s, u * s + v * c], -1).flatten(-2)


def _owners(offsets, T):
    """(request, index within the request) of every token."""
    t = torch.arange(T, device=offsets.device)
    b = torch.searchsorted(offsets[1:].long(), t, right=True)
    return b, t - offsets.long()[b]


def _slots(s, T):
    """Flat cache rows of the step's tokens, and their places in their requests."""
    b, i = _owners(s["offsets"], T)
    off = s["offsets"].long()
    place = (s["seq_lens"].long() - (off[1:] - off[:-1]))[b] + i
    return s["block_table"].long()[b, place // PAGE] * PAGE + place % PAGE, place


def _plain_query(s):
    q = s["q"].float()
    lat = torch.bmm(q[..., :DN].transpose(0, 1), s["w_uk"].float()).transpose(0, 1)
    return lat.to(torch.bfloat16).contiguous(), _turn(q[..., DN:], s["positions"], s["rate"]).to(torch.bfloat16)


def _plain_append(s):
    kv = s["kv"].float()
    at, place = _slots(s, kv.shape[0])
    c = kv[:, :DL]
    c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["gamma"].float()
    k = _turn(kv[:, DL:], place if s["positions"] is None else s["positions"], s["rate"])
    rows = torch.cat([c, k], -1)
    cache = s["cache"]
    flat = cache.view(-1, cache.shape[-1])
    flat[at] = _quantise(rows) if cache.dtype == torch.uint8 else rows.to(torch.bfloat16)
    return _held(cache) if cache.dtype == torch.uint8 else cache


def _plain_tree(s):
    T, B, N = s["q_latent"].shape[0], s["seq_lens"].shape[0], s["most"]
    off = s["offsets"].long()
    counts = off[1:] - off[:-1]
    n = torch.arange(N, device=off.device)
    pick = (off[:-1, None] + n).clamp(max=T - 1)                                   # [B][N]
    q = torch.cat([s["q_latent"], s["q_rope"]], -1).float()[pick].view(B, N * H, ROW)
    kv = _rows(s["cache"][s["block_table"].long().clamp(min=0)]).view(B, -1, ROW)  # [B][keys][576]
    prefix = (s["seq_lens"].long() - counts)[:, None, None]
    key = torch.arange(kv.shape[1], device=off.device)
    bit = (key - prefix).clamp(0, 63)
    seen = (key < prefix) | ((s["masks"][pick][..., None] >> bit & 1).bool() & (key < prefix + counts[:, None, None]))
    x = torch.baddbmm(torch.zeros((), device=q.device), q, kv.transpose(1, 2), beta=0, alpha=SCALE).view(B, N, H, -1)
    x.masked_fill_(~seen[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = x.sum(-1)
    o = torch.bmm(x.view(B, N * H, -1), kv[..., :DL]).view(B, N, H, DL) / total.clamp(min=1e-30)[..., None]
    lse = m[..., 0] + total.log()
    b, i = _owners(s["offsets"], T)
    return o[b, i].to(torch.bfloat16), lse[b, i]


def _plain_commit(s):
    cache = s["cache"]
    flat = cache.view(cache.shape[0], -1, cache.shape[-1])
    off = s["offsets"].long()
    prefix = s["seq_lens"].long() - (off[1:] - off[:-1])
    i = torch.arange(s["paths"].shape[1], device=off.device)
    there = i < s["path_lens"].long()[:, None]
    to = prefix[:, None] + i
    of = torch.where(there, prefix[:, None] + s["paths"].long(), to)
    table = s["block_table"].long()

    def slot(p):
        p = torch.where(there, p, prefix[:, None])        # a request accepts its root at least
        return table.gather(1, p // PAGE) * PAGE + p % PAGE

    to, of = slot(to), slot(of)
    flat[:, to] = flat[:, of]
    held = _held(cache) if cache.dtype == torch.uint8 else (cache,)
    return held + ((prefix + s["path_lens"]).to(torch.int32),)


# ------------------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if not own:
        return {"query": _plain_query, "append": _plain_append, "tree": _plain_tree, "commit": _plain_commit}[op](s)
    import mla_decode_attention_02_gb300 as mla
    if op == "query":
        q_latent, q_rope, _ = mla.query(s["q"][..., :DN], s["q"][..., DN:], s["w_uk"], s["positions"], table=s["table"], status=s["status"])
        return q_latent, q_rope
    cache = s["cache"]
    fp8 = cache.dtype == torch.uint8
    if op == "append":
        append = mla.cache_append_fp8 if fp8 else mla.cache_append
        append(s["kv"][:, :DL], s["kv"][:, DL:], s["gamma"], cache, s["block_table"], s["seq_lens"], s["offsets"],
               positions=s["positions"], table=s["table"], rms_eps=EPS, status=s["status"])
        return _held(cache) if fp8 else cache
    if op == "tree":
        p = mla.tree_plan(s["seq_lens"], s["offsets"], s["masks"], max_pages_per_seq=s["block_table"].shape[1])
        decode = mla.tree_decode_fp8 if fp8 else mla.tree_decode
        return decode(p, s["q_latent"], s["q_rope"], cache, s["block_table"], scale=SCALE)
    commit = mla.cache_commit_fp8 if fp8 else mla.cache_commit
    new_lens, _ = commit(cache, s["block_table"], s["seq_lens"], s["offsets"], s["paths"], s["path_lens"], status=s["status"])
    return (_held(cache) if fp8 else (cache,)) + (new_lens,)


# ------------------------------------------------------------------------------ in 64 bits

def _rotate64(x, positions):
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    z = torch.view_as_complex(x.double().reshape(x.shape[:-1] + (DR // 2, 2)).contiguous())
    i = torch.arange(DR // 2, dtype=torch.float64, device=x.device)
    angle = positions.double()[:, None] * torch.exp(i * (-2.0 * math.log(BASE) / DR))
    turn = torch.polar(torch.ones_like(angle), angle).view((x.shape[0],) + (1,) * (x.dim() - 2) + (DR // 2,))
    out.copy_(torch.view_as_real(z * turn).reshape(x.shape))
    return out


def _e4m3_64(x):
    """The e4m3 values nearest to x (ties to even, saturating), in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    if case["op"] == "commit":
        return None                                        # rows are moved, nothing is computed
    s = prepare(case, seed)
    if case["op"] == "query":
        q = s["q"].double()
        return torch.einsum("thk,hkn->thn", q[..., :DN], s["w_uk"].double()), _rotate64(q[..., DN:], s["positions"])
    counts, lengths = _sizes(case)
    table = s["block_table"].cpu().tolist()
    if case["op"] == "append":
        slots, places = [], []
        for b, (c, L) in enumerate(zip(counts, lengths)):
            for p in range(L - c, L):
                slots.append(table[b][p // PAGE] * PAGE + p % PAGE)
                places.append(p)
        places = torch.tensor(places, device="cuda") if s["positions"] is None else s["positions"]
        x = s["kv"].double()
        norm = torch.linalg.vector_norm(x[:, :DL], dim=1, keepdim=True)
        c = x[:, :DL] / torch.sqrt(norm * norm / DL + EPS) * s["gamma"].double()
        k = _rotate64(x[:, DL:], places)
        at = torch.tensor(slots, device="cuda")
        shape = s["cache"].shape[:2]

        def spread(v):
            full = torch.zeros((shape[0] * shape[1], v.shape[1]), dtype=torch.float64, device="cuda")
            full[at] = v
            return full.view(shape + (v.shape[1],))

        if not case["fp8"]:
            return spread(torch.cat([c, k], 1))
        size = c.abs().amax(1, keepdim=True) / E4M3_MAX
        return spread(_e4m3_64(c / size)), spread(k / size), spread(size)
    o, lse = [], []
    masks = s["masks"].cpu().tolist()
    t = 0
    for b, (c, L) in enumerate(zip(counts, lengths)):
        if c == 0:
            continue
        keys = s["cache"][s["block_table"][b, :(L + PAGE - 1) // PAGE].long()]
        if case["fp8"]:
            code, rope, size = _held(keys)
            keys = torch.cat([code.double(), rope.double()], -1) * size.double()
        keys = keys.double().reshape(-1, ROW)[:L]
        for i in range(c):
            seen = torch.ones(L, dtype=torch.bool)
            seen[L - c:] = torch.tensor([bool(masks[t] >> j & 1) for j in range(c)])
            seen = seen.cuda()
            q = torch.cat([s["q_latent"][t], s["q_rope"][t]], 1).double()
            x = torch.where(seen, (q @ keys.T) * SCALE, -math.inf)
            o.append(torch.softmax(x, 1) @ keys[:, :DL])
            lse.append(torch.logsumexp(x, 1))
            t += 1
    return torch.stack(o), torch.stack(lse)
