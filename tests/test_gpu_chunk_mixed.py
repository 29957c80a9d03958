"""Chunks whose requests do not all suit one form: the plan takes one for each, and a slot that does nothing changes nothing.

The rows of a request in the form with per-head keys do not depend on the batch around it (its tiles, keys and sums are its
own), so they are compared bit for bit with the request alone.  The absorbed form's rows are held to the bound of
test_gpu_chunk.py (6e-3 of the norm, a row three times that; its derivation is there).
"""

import numpy as np
import pytest
import torch

import chunk_util as CU
import mla_decode_attention_02_gb300 as mla
import oracle.chunk as OC

pytestmark = pytest.mark.gpu
SCALE = mla.DEFAULT_SCALE
PICK = [0, 77, 127]


def plan(c, **kw):
    kw.setdefault("kv_tokens", c["kv_tokens"])
    return mla.chunk_plan(c["seq_lens"], c["offsets"], tokens=c["T"], max_pages_per_seq=c["block_table"].shape[1], **kw)


def attend(c, p=None, **kw):
    f = mla.chunk_attend_fp8 if c["cache"].dtype == torch.uint8 else mla.chunk_attend
    return f(p or plan(c), c["q"][..., :128], c["q"][..., 128:], c["w_uk"], c["w_uv"], c["cache"], c["block_table"],
             scale=SCALE, **kw)


def equal(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def alone(c, b):
    """Request b of a case as a step of its own."""
    off = c["offsets"].tolist()
    L = int(c["seq_lens"][b])
    t = slice(off[b], off[b + 1])
    return dict(c, T=off[b + 1] - off[b], n=off[b + 1] - off[b], counts=[off[b + 1] - off[b]], q=c["q"][t].contiguous(),
                kv_tokens=-(-L // 64) * 64, seq_lens=c["seq_lens"][b:b + 1].clone(), block_table=c["block_table"][b:b + 1].clone(),
                offsets=torch.tensor([0, off[b + 1] - off[b]], dtype=torch.int32, device="cuda"))


def forms(p):
    """Of a mixed plan, whether each request is in the absorbed form."""
    tiles = p.tokens // 256 + min(p.batch, p.tokens) + 1
    at = (64 + 32 * tiles + 8 * (p.kv_tokens // 64) + 255) // 256 * 256
    return p.workspace[at:at + p.batch].bool().tolist()


def whole(n, L, units):
    return L * (248 + 50 * ((n + 127) // 128)) // 10 + 4550 * ((n + 255) // 256) * 128 // (2 * units)


def absorbed(n, L, units):
    return 34 * n + 1044 * n * (L + 7 * 64) // (64 * units)


def gain(n, L, units):
    return whole(n, L, units) * 3 // 4 - absorbed(n, L, units)


def expected(counts, lens):
    units = mla.num_units()
    g = [gain(n, L, units) if n else 0 for n, L in zip(counts, lens)]
    keeps = any(n and x <= 0 for n, x in zip(counts, g))
    return keeps, sum(x for x in g if x > 0), g


def close(c, out, lse, rows):
    o, l, _, _ = OC.chunk_attend(c["q"][:, PICK], c["w_uk"][PICK], c["w_uv"][PICK], c["cache"], c["block_table"],
                                 c["seq_lens"].tolist(), c["offsets"].tolist(), scale=SCALE)
    o, l, got = o[rows], l[rows], out[rows][:, PICK].double()
    off, size = (got - o).norm(dim=-1), o.norm(dim=-1)
    assert off.norm() <= 6e-3 * size.norm() and (off <= 1.8e-2 * size).all(), (off.norm() / size.norm(), (off / size).max())
    assert (lse[rows][:, PICK].double() - l).abs().max() <= 2.0 ** -8 * SCALE * 512


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("tokens,keys", [(512, 12000), (300, 30000), (1, 20000)])
@pytest.mark.parametrize("idle", [1, 31, 300])
def test_idle_slots_change_nothing(tokens, keys, idle, fp8):
    """One request among slots without tokens: the form, and so the bits, of the request alone."""
    at = idle // 3
    counts = [0] * at + [tokens] + [0] * (idle - at)
    lens = [(7 * i) % 5000 for i in range(at)] + [keys] + [10 ** 9] * (idle - at)
    c = CU.case(counts, lens, seed=71, fp8=fp8, pad=3 if tokens > 80 else 100)
    p = plan(c)
    lse = torch.full((c["T"], 128), 7.0, device="cuda")
    out = torch.full((c["T"], 128, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    attend(c, p, out=out, lse=lse)
    assert mla.check(p) == 0
    assert (out[tokens:] == 7).all() and (lse[tokens:] == 7).all()
    one = alone(c, at)
    ref_lse = torch.empty(tokens, 128, device="cuda")
    ref = attend(one, lse=ref_lse)
    if tokens > 80:
        assert forms(p) == [False] * (idle + 1)
        assert equal(out[:tokens], ref) and torch.equal(lse[:tokens], ref_lse)
    else:      # few tokens, much padding
        assert forms(p) == [i == at for i in range(idle + 1)]
        close(c, out, lse, slice(0, tokens))


# a long chunk beside requests of a few tokens over long contexts, one of each kind among idle slots
COUNTS = [2, 0, 300, 1, 40, 0, 1, 400, 3, 0]
LENS = [5000, 70, 3000, 6400, 5001, 0, 64, 400, 7000, 10 ** 9]
FORMS = [True, False, False, True, True, False, True, False, True, False]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_a_form_for_each_request(fp8):
    c = CU.case(COUNTS, LENS, seed=72, fp8=fp8, pad=5)
    keeps, saved, g = expected(COUNTS, LENS)
    assert keeps and saved > 36000 + 10 * c["T"] and [x > 0 for x in g] == FORMS
    p = plan(c)
    out = torch.full((c["T"], 128, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c["T"], 128), 7.0, device="cuda")
    attend(c, p, out=out, lse=lse)
    assert mla.check(p) == 0 and forms(p) == FORMS
    assert (out[c["n"]:] == 7).all() and (lse[c["n"]:] == 7).all()
    close(c, out, lse, slice(0, c["n"]))
    off = c["offsets"].tolist()
    for b in (2, 7):
        one = alone(c, b)
        ref_lse = torch.empty(one["T"], 128, device="cuda")
        assert equal(attend(one, lse=ref_lse), out[off[b]:off[b + 1]]) and torch.equal(ref_lse, lse[off[b]:off[b + 1]])
    again = attend(c, p)                                   # without lse, and once more
    assert equal(again[:c["n"]], out[:c["n"]])
    # passes over the heads, and without room for expanded pages: the same values of the one form, close ones of the other
    full = mla.chunk_scratch_size(p, 128, fp8=fp8)
    rows = torch.cat([torch.arange(off[b], off[b + 1]) for b in (2, 7)]).cuda()
    for heads in (1, 50):
        room = torch.full((mla.chunk_scratch_size(p, heads, fp8=fp8),), 0xFF, dtype=torch.uint8, device="cuda")
        assert room.numel() < full
        assert equal(attend(c, p, scratch=room)[:c["n"]], out[:c["n"]])
    if fp8:
        least = mla.chunk_scratch_size(p, 1)
        room = torch.full((least,), 0xFF, dtype=torch.uint8, device="cuda")
        thin = attend(c, p, scratch=room, lse=lse)
        close(c, thin, lse, slice(0, c["n"]))
        assert equal(thin[rows], out[rows])
        with pytest.raises(mla.MLAError):
            attend(c, p, scratch=room[:least - 1])


def test_the_choice_follows_its_rule():
    """Ragged steps of all kinds, more requests than the planner scans at a time among them."""
    rng = np.random.default_rng(73)
    units, mixed = mla.num_units(), 0
    for trial in range(40):
        B = int(rng.choice([2, 5, 30, 1100, 2500]))
        counts = [int(2 ** rng.uniform(0, 9 if B < 100 else 3)) if rng.random() < 0.7 else 0 for _ in range(B)]
        lens = [max(n, int(2 ** rng.uniform(4, 14 if B < 100 else 8))) for n in counts]
        bad = int(rng.integers(B)) if trial % 4 == 0 else -1
        if bad >= 0 and counts[bad]:
            lens[bad] = counts[bad] - 1
        T, kv = sum(counts), sum(-(-L // 64) * 64 for n, L in zip(counts, lens) if n)
        if not 80 < T < 9000:
            continue
        width = 1 << 15
        p = mla.chunk_plan(torch.tensor(lens, dtype=torch.int32, device="cuda"),
                           torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda"),
                           tokens=T, max_pages_per_seq=width, kv_tokens=kv)
        if whole(1, kv, units) < 400000 or (T <= 256 and 36000 + absorbed(T, min(kv, width * 64), units) < 3 * whole(1, kv, units)):
            continue                                         # (may be one form for the step)
        k, saved, g = expected([0 if i == bad else n for i, n in enumerate(counts)], lens)
        k = k or (bad >= 0 and counts[bad] > 0)
        take = saved > 36000 + 10 * T - (0 if k else 14250)
        assert forms(p) == [take and x > 0 for x in g], (trial, B, T, kv)
        assert bool(mla.check(p) & mla.MLA_DEV_BAD_SEQ_LEN) == (bad >= 0 and counts[bad] > 0)
        mixed += take
    assert mixed >= 10


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_bad_inputs_of_either_form(fp8):
    c = CU.case(COUNTS, LENS, seed=74, fp8=fp8, pad=2)
    ref, n, off = attend(c), c["n"], c["offsets"].tolist()

    def spoilt(d, status, which):
        p = plan(d)
        out = torch.full((d["T"], 128, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        attend(d, p, out=out)
        assert mla.check(p) & status, (status, mla.check(p))
        for b in range(len(COUNTS)):
            t = slice(off[b], off[b + 1])
            if b in which:
                assert torch.isnan(out[t].float()).all(), b
            elif FORMS[b]:      # (another cut of the same keys)
                assert (out[t].double() - ref[t].double()).norm() <= 1.2e-2 * ref[t].double().norm(), b
            else:
                assert equal(out[t], ref[t]), b
        assert (out[n:] == 7).all()

    for b in (0, 2, 4):                                      # a page outside the pool: a request in each form
        d = dict(c, block_table=c["block_table"].clone())
        d["block_table"][b, 1] = -1 if b else 1 << 30
        spoilt(d, mla.MLA_DEV_BAD_PAGE, [b])
    for b in (2, 8):                                         # a length below its tokens (then in the form with keys) or beyond the table
        for bad in (COUNTS[b] - 1, -5, 64 * c["block_table"].shape[1] + 1):
            d = dict(c, seq_lens=c["seq_lens"].clone())
            d["seq_lens"][b] = bad
            spoilt(d, mla.MLA_DEV_BAD_SEQ_LEN, [b])
    for bad in ([1] + off[1:], off[:3] + [off[-1] + 5] + off[4:], off[:-1] + [c["T"] + 1], [0] + [-3] + off[2:]):
        d = dict(c, offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        p = plan(d)
        out = attend(d, p, lse=torch.zeros(c["T"], 128, device="cuda"))
        assert mla.check(p) & mla.MLA_DEV_BAD_OFFSETS and torch.isnan(out.float()).all()


def test_more_pages_than_said():
    """Fewer keys than the requests of the one form hold: their tokens are NaN; the absorbed form's do not depend on it."""
    counts, lens = [600] + [1] * 12, [11000] + [2000] * 12
    c = CU.case(counts, lens, seed=78)
    p = plan(c)
    ref = attend(c, p)
    assert mla.check(p) == 0 and forms(p) == [False] + [True] * 12
    p = plan(c, kv_tokens=10240)
    out = attend(c, p)
    assert mla.check(p) & mla.MLA_DEV_BAD_KV_TOKENS and torch.isnan(out[:600].float()).all() and equal(out[600:], ref[600:])


@pytest.mark.parametrize("field", ["tokens", "max_pages", "batch"])
def test_another_plan_in_the_workspace(field):
    c = CU.case(COUNTS, LENS, seed=75, spare=0)
    p = plan(c)
    setattr(p, field, getattr(p, field) - 1)
    d = dict(c, q=c["q"][:p.tokens], block_table=c["block_table"][:p.batch, :p.max_pages].contiguous())
    out = torch.full((p.tokens, 128, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.tokens, 128), 7.0, device="cuda")
    attend(d, p, out=out, lse=lse)
    assert mla.check(p) & mla.MLA_DEV_BAD_PLAN and (out == 7).all() and (lse == 7).all()


def test_what_is_not_seen_counts_nothing_in_either_form():
    """The last tokens of a request of each form hold infinity and NaN."""
    c = CU.case(COUNTS, LENS, seed=76)
    ref, off = attend(c), c["offsets"].tolist()
    hold = {(2, LENS[2] - 1): float("nan"), (4, LENS[4] - 1): float("inf")}
    out = attend(CU.case(COUNTS, LENS, seed=76, hold=hold))
    last = [off[3] - 1, off[5] - 1]
    rest = [t for t in range(c["n"]) if t not in last]
    assert equal(out[rest], ref[rest]) and torch.isnan(out[last].float()).all()


def test_a_captured_step_whose_requests_change_forms():
    """Replays of one graph: long chunks and single tokens change places, one form takes all, the other does, none has tokens."""
    steps = [(COUNTS, LENS), (COUNTS[::-1], LENS[::-1]), ([100, 0, 100, 100, 0, 0, 100, 100, 100, 0], [900] * 10),
             ([3] * 10, [4000] * 10), ([0] * 10, [5] * 10), (COUNTS, LENS)]
    width, T, pages = 128, sum(COUNTS) + 3, 700
    seq_lens, offsets = torch.zeros(10, dtype=torch.int32, device="cuda"), torch.zeros(11, dtype=torch.int32, device="cuda")
    table = torch.zeros(10, width, dtype=torch.int32, device="cuda")
    base = CU.case([1], [1], seed=77)
    q, cache = torch.zeros(T, 128, 192, dtype=torch.bfloat16, device="cuda"), torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    d = dict(base, T=T, seq_lens=seq_lens, offsets=offsets, block_table=table, q=q, cache=cache, kv_tokens=30016)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        attend(d, plan(d))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            p = plan(d)
            out = attend(d, p)
    for i, (counts, lens) in enumerate(steps):
        e = CU.case(counts, lens, seed=80 + i, pad=T - sum(counts), width=width)
        seq_lens.copy_(e["seq_lens"])
        offsets.copy_(e["offsets"])
        table.copy_(e["block_table"])
        q.copy_(e["q"])
        cache[:e["cache"].shape[0]] = e["cache"]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert mla.check(p) == 0
        f = dict(e, w_uk=base["w_uk"], w_uv=base["w_uv"], kv_tokens=30016)
        r = plan(f)
        assert equal(out[:sum(counts)], attend(f, r)[:sum(counts)]), i
        assert forms(p) == forms(r)
        if i in (0, 5):
            assert forms(p) == FORMS
        elif sum(counts):
            lse = torch.empty(T, 128, device="cuda")
            close(f, attend(f, lse=lse), lse, slice(0, sum(counts)))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_layers_behind_one_another(fp8):
    """Mixed steps with what follows them in a layer at once behind: each kernel may start before the one ahead is done, and
    takes tensor memory of its own; the results are those of steps with a pause between."""
    c = CU.case(COUNTS, LENS, seed=90, fp8=fp8)
    none = CU.case([200, 100, 0, 300], [900, 3000, 70, 7000], seed=91, fp8=fp8)          # (no request in the absorbed form)
    g = torch.Generator(device="cuda").manual_seed(92)
    w_o = (torch.randn(1024, 16384, generator=g, device="cuda") / 128).to(torch.bfloat16)
    table = mla.rope_table()

    def layer(d, p, wait):
        o = attend(d, p)
        if wait:
            torch.cuda.synchronize()
        out = mla.epilog_oproj(o, w_o)
        ql, _, _ = mla.query(d["q"][..., :128], d["q"][..., 128:], d["w_uk"], torch.zeros(d["T"], dtype=torch.int32, device="cuda"),
                             table=table)
        return o, out, ql

    plans = [(d, plan(d)) for d in (c, none)]
    assert forms(plans[0][1]) == FORMS and not any(forms(plans[1][1]))
    refs = []
    for d, p in plans:
        refs.append([x.clone() for x in layer(d, p, True)])
        torch.cuda.synchronize()
    outs = [layer(d, p, False) for _ in range(4) for d, p in plans]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs += [layer(d, p, False) for _ in range(2) for d, p in plans]
    graph.replay()
    torch.cuda.synchronize()
    for i, got in enumerate(outs):
        for a, b in zip(got, refs[i % 2]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)), i
    assert all(mla.check(p) == 0 for _, p in plans)
