"""GPU parity of attention over chunks of prompts with the 64-bit oracle.

Tolerances, from the roundings (a bf16 rounding is off by at most BF = 2^-8 of the value, by 2^-8 / sqrt(3) in the
mean square at most), for inputs N(0, 1), W ~ N(0, 1 / 512), so that k, v and q are of size 1:

* a key's rounding moves a score by at most d = BF * reach (reach = scale sum |q k| over the 128 no-position dims; the
  rotary part is as stored, for an fp8 cache rounded once more: BF again on 64 dims), fp32 sums by 1e-4; a weight so
  moves by at most 2 d (its own score and the sum), and lse by d.
* the weights are rounded once, the values once, the output once:
  |o - ref| <= (2 d + 2 BF) spread + BF |ref| + 1e-6, and |lse - ref| <= d.
* these are independent, and in the mean square each is at most BF / sqrt(3) = 2.25e-3 of o (values, weights, output),
  a score's scale sqrt(sum q^2 k^2) BF / sqrt(3) = 0.82 BF / sqrt(3) = 1.9e-3: together at most 4.4e-3 of o's norm; of one
  row's norm three times that (128 values of one row share their weights).
"""

import math

import numpy as np
import pytest
import torch

import chunk_util as CU
import mla_decode_attention_02_gb300 as mla
import oracle.chunk as OC

pytestmark = pytest.mark.gpu
SCALE = mla.DEFAULT_SCALE
BF = 2.0 ** -8


def plan(c, **kw):
    kw.setdefault("kv_tokens", c["kv_tokens"])
    return mla.chunk_plan(c["seq_lens"], c["offsets"], tokens=c["T"], max_pages_per_seq=c["block_table"].shape[1], **kw)


def attend(c, p=None, **kw):
    f = mla.chunk_attend_fp8 if c["cache"].dtype == torch.uint8 else mla.chunk_attend
    return f(p or plan(c), c["q"][..., :128], c["q"][..., 128:], c["w_uk"], c["w_uv"], c["cache"], c["block_table"],
             scale=SCALE, **kw)


def check(c, out, lse=None, rows=None, what=""):
    o, l, spread, reach = OC.chunk_attend(c["q"], c["w_uk"], c["w_uv"], c["cache"], c["block_table"], c["seq_lens"].tolist(),
                                          c["offsets"].tolist(), scale=SCALE)
    rows = slice(0, c["n"]) if rows is None else rows
    o, l, spread, reach, got = o[rows], l[rows], spread[rows], reach[rows], out[rows].double()
    assert torch.isfinite(got).all(), what
    extra = SCALE * BF * c["q"][rows][..., 128:].double().norm(dim=-1) * 14 if c["cache"].dtype == torch.uint8 else 0.0
    d = BF * reach + extra + 1e-4      # (14: beyond the largest norm of 64 N(0, 1) values)
    over = (got - o).abs() - ((2 * d + 2 * BF)[..., None] * spread + BF * o.abs() + 1e-6)
    assert over.max() <= 0, f"{what}: o beyond its bound by {over.max():.3e}"
    off, size = (got - o).norm(dim=-1), o.norm(dim=-1)
    assert off.norm() <= 4.4e-3 * size.norm(), f"{what}: {off.norm() / size.norm():.3e} of the norm"
    assert (off <= 1.3e-2 * size).all(), f"{what}: a row {(off / size).max():.3e} of its norm"
    if lse is not None:
        assert ((lse[rows].double() - l).abs() <= d).all(), what


CASES = [
    # counts, lens
    ([1], [1]),                                    # one token, no context
    ([1], [64]),
    ([2], [130]),
    ([127], [127]),
    ([128], [128]),                                # whole tiles
    ([129], [200]),
    ([256], [256]),
    ([257], [1000]),                               # two tiles, the second of one token
    ([64], [65]),
    ([1, 1, 1], [63, 64, 65]),
    ([100, 0, 3, 300, 0], [700, 0, 3, 301, 10 ** 9]),   # slots of the batch without tokens
    ([511, 77], [600, 1500]),
    ([700], [700]),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("counts,lens", CASES, ids=[f"{i}" for i in range(len(CASES))])
def test_parity(counts, lens, fp8):
    c = CU.case(counts, lens, seed=3, pad=3, fp8=fp8)
    p = plan(c)
    out = torch.full((c["T"], 128, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c["T"], 128), 7.0, device="cuda")
    assert attend(c, p, out=out, lse=lse) is out
    assert mla.check(p) == 0
    check(c, out, lse)
    assert (out[c["n"]:] == 7).all() and (lse[c["n"]:] == 7).all()      # rows behind the last request
    again = attend(c, p)                                                  # the plan serves another call, without lse
    assert torch.equal(again[:c["n"]], out[:c["n"]])


# A form is chosen by its expected time; these take the absorbed one (few tokens, long contexts) ...
ABSORBED = [([3], [3000]), ([1, 0, 40, 7], [5000, 0, 3001, 2048]), ([65, 70], [9000, 6400])]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("counts,lens", ABSORBED, ids=[f"{i}" for i in range(len(ABSORBED))])
def test_few_tokens_over_long_contexts(counts, lens, fp8):
    """Roundings of the absorbed form: queries, weights, latent outputs and outputs once in bf16.

    The queries move a score by at most BF scale sum |q_latent c| over 512 values (their mean square: BF / sqrt(3)
    of 0.82); weights (rounded twice at most), latent outputs and outputs make 2.25e-3 of o each (weights twice
    that), and the projection sums 512 rounded values: in the mean square below 6e-3 of o's norm altogether, a row three times that.
    """
    c = CU.case(counts, lens, seed=5, pad=2, fp8=fp8)
    p = plan(c)
    out = torch.full((c["T"], 128, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c["T"], 128), 7.0, device="cuda")
    attend(c, p, out=out, lse=lse)
    assert mla.check(p) == 0
    check_absorbed(c, out, lse)
    assert (out[c["n"]:] == 7).all() and (lse[c["n"]:] == 7).all()


def check_absorbed(c, out, lse=None):
    o, l, _, _ = OC.chunk_attend(c["q"], c["w_uk"], c["w_uv"], c["cache"], c["block_table"], c["seq_lens"].tolist(),
                                 c["offsets"].tolist(), scale=SCALE)
    n = c["n"]
    off, size = (out[:n].double() - o[:n]).norm(dim=-1), o[:n].norm(dim=-1)
    assert off.norm() <= 6e-3 * size.norm() and (off <= 1.8e-2 * size).all(), (off.norm() / size.norm(), (off / size).max())
    if lse is not None:
        # sum |q_latent c| over 512 products of a normal q_latent of size 1 / sqrt(2) ... 0.82 and a normal c: below 512
        assert (lse[:n].double() - l[:n]).abs().max() <= BF * SCALE * 512


def equal(a, b, n):
    return torch.equal(a[:n].view(torch.int16), b[:n].view(torch.int16))


WHOLE = ([100, 0, 300, 128], [700, 0, 301, 400])      # (many tokens for their keys: the form with per-head keys)
FEW = ([3, 0, 20], [3000, 0, 2500])


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("shape", [WHOLE, FEW], ids=["whole", "few"])
def test_what_is_not_seen_counts_nothing(shape, fp8):
    """NaN and infinities in slots past the end, in spare pages, in other requests and in a chunk's later tokens."""
    counts, lens = shape
    c = CU.case(counts, lens, seed=7, fp8=fp8)
    ref = attend(c)
    # the last request's last two tokens are spoilt: those two see NaN, all before see what they saw
    L = lens[-1]
    hold = {(len(counts) - 1, L - 2): float("inf"), (len(counts) - 1, L - 1): float("nan")}
    d = CU.case(counts, lens, seed=7, fp8=fp8, hold=hold)
    out = attend(d)
    n = c["n"]
    assert equal(out, ref, n - 2)
    assert torch.isnan(out[n - 2:n].float()).all()


def test_a_spoilt_rotary_part_spoils_what_sees_it():
    c = CU.case([130], [200], seed=8)
    row = c["block_table"][0, 150 // 64]
    ref = attend(c)
    c["cache"][int(row), 150 % 64, 512 + 5] = float("nan")
    out = attend(c)
    at = 150 - 70                                          # the token of slot 150
    assert equal(out, ref, at) and torch.isnan(out[at:].float()).all()


@pytest.mark.parametrize("shape", [WHOLE, FEW], ids=["whole", "few"])
def test_bad_pages_lengths_and_offsets(shape):
    counts, lens = shape
    c = CU.case(counts, lens, seed=9, pad=1)
    ref = attend(c)
    n, off = c["n"], c["offsets"].tolist()
    # a page outside the pool: the request's tokens that see it
    for page in (-1, int(c["cache"].shape[0]), 1 << 30):
        d = dict(c, block_table=c["block_table"].clone())
        d["block_table"][0, 1] = page
        p = plan(d)
        out = attend(d, p)
        assert mla.check(p) & mla.MLA_DEV_BAD_PAGE
        assert torch.isnan(out[:off[1]].float()).all() and equal(out[off[1]:], ref[off[1]:], n - off[1])
    # a length below its tokens, or beyond the table
    for bad in (counts[0] - 1, -5, 64 * c["block_table"].shape[1] + 1):
        d = dict(c, seq_lens=c["seq_lens"].clone())
        d["seq_lens"][0] = bad
        p = plan(d)
        out = attend(d, p)
        assert mla.check(p) & mla.MLA_DEV_BAD_SEQ_LEN
        assert torch.isnan(out[:off[1]].float()).all() and equal(out[off[1]:], ref[off[1]:], n - off[1])
    # offsets that are none: every row
    for bad in ([1] + off[1:], off[:1] + [off[-1] + 5] + off[2:], off[:-1] + [c["T"] + 1], [0] + [-3] + off[2:]):
        d = dict(c, offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        p = plan(d)
        out = attend(d, p, lse=torch.zeros(c["T"], 128, device="cuda"))
        assert mla.check(p) & mla.MLA_DEV_BAD_OFFSETS
        assert torch.isnan(out.float()).all()


def test_more_pages_than_said():
    c = CU.case([100, 40], [700, 300], seed=10)
    p = plan(c, kv_tokens=c["kv_tokens"] - 64)
    out = attend(c, p)
    assert mla.check(p) & mla.MLA_DEV_BAD_KV_TOKENS and torch.isnan(out.float()).all()


def test_no_tokens_at_all():
    c = CU.case([0, 0], [0, 70], seed=11, pad=5)
    p = plan(c, kv_tokens=128)
    out = torch.full((5, 128, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    attend(c, p, out=out)
    assert mla.check(p) == 0 and (out == 7).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_passes_over_the_heads_change_no_bit(fp8):
    c = CU.case([300, 90], [900, 500], seed=12, fp8=fp8)
    p = plan(c)
    ref = attend(c, p)
    for heads in (1, 5, 64, 127):
        room = torch.full((mla.chunk_scratch_size(p, heads, fp8=fp8),), 0xFF, dtype=torch.uint8, device="cuda")
        assert equal(attend(c, p, scratch=room), ref, c["n"])      # (0xFF: NaN in whatever is not written)


def test_a_loose_bound_and_a_wide_table_change_no_bit():
    c = CU.case([300, 90], [900, 500], seed=13)
    ref = attend(c)
    wide = CU.case([300, 90], [900, 500], seed=13, width=40)
    assert equal(attend(wide, plan(wide, kv_tokens=None)), ref, c["n"])


@pytest.mark.parametrize("scale", [4.0, 30.0])
def test_large_and_rising_scores(scale):
    """Maxima that grow from key tile to key tile, so that the reference is raised and the outputs rescaled."""
    c = CU.case([200, 60], [900, 700], seed=14)
    c["q"] *= scale
    grow = torch.linspace(0.2, 3.0, 900, device="cuda")
    for b, L in enumerate((900, 700)):
        for j in range(-(-L // 64)):
            part = c["cache"][int(c["block_table"][b, j])]
            part *= grow[j * 64:j * 64 + 64][:part.shape[0], None].to(torch.bfloat16) if (j + 1) * 64 <= 900 else 1
    out = attend(c)
    o, _, spread, reach = OC.chunk_attend(c["q"], c["w_uk"], c["w_uv"], c["cache"], c["block_table"], [900, 700],
                                          c["offsets"].tolist(), scale=SCALE)
    # scores of size 100: fp32 sums of 192 products are off by 192 2^-24 of sum |q k|, the shift by 2^-24 of a score
    d = BF * reach + 2e-5 * reach + 1e-4
    over = (out.double() - o).abs() - ((torch.exp(2 * d) - 1 + 2 * BF)[..., None] * spread * 2 + BF * o.abs() + 1e-6)
    assert torch.isfinite(out.float()).all() and over.max() <= 0, over.max()


def test_strided_queries_and_another_stream():
    c = CU.case([150, 70], [600, 200], seed=15)
    ref = attend(c)
    wide = torch.zeros(c["T"], 130, 256, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:129, 8:200] = c["q"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p = mla.chunk_plan(c["seq_lens"], c["offsets"], tokens=c["T"], max_pages_per_seq=c["block_table"].shape[1],
                       kv_tokens=c["kv_tokens"], stream=s)
    out = mla.chunk_attend(p, wide[:, 1:129, 8:136], wide[:, 1:129, 136:200], c["w_uk"], c["w_uv"], c["cache"], c["block_table"],
                           scale=SCALE, stream=s)
    s.synchronize()
    assert equal(out, ref, c["n"])


@pytest.mark.parametrize("shape", [WHOLE, FEW], ids=["whole", "few"])
def test_captured_step_follows_its_inputs(shape):
    """Plan and attention in a graph: replays read the lengths, offsets and values of the moment."""
    counts, lens = shape
    c = CU.case(counts, lens, seed=16, pad=4)
    static = {k: c[k].clone() for k in ("seq_lens", "offsets", "q", "cache", "block_table")}
    d = dict(c, **static)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        attend(d, plan(d))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            p = plan(d)
            out = attend(d, p)
    for seed, cut in ((16, 0), (17, 1)):
        other = [max(n - cut, 0) for n in counts]
        e = CU.case(other, [L - cut if n else 0 for n, L in zip(counts, lens)], seed=seed, width=c["block_table"].shape[1],
                    pad=c["T"] - sum(other))
        for k, v in static.items():
            v.copy_(e[k][:v.shape[0]] if k != "cache" else torch.nn.functional.pad(
                e[k], (0, 0, 0, 0, 0, max(0, v.shape[0] - e[k].shape[0])))[:v.shape[0]])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        f = dict(e, kv_tokens=c["kv_tokens"], w_uk=c["w_uk"], w_uv=c["w_uv"])
        assert equal(out, attend(f, plan(f)), sum(other)), seed


def test_two_steps_at_once():
    """Two plans on two streams, each with its own workspace and scratch."""
    cs = [CU.case([500, 30], [800, 700], seed=18), CU.case([256], [1000], seed=19)]
    refs = [attend(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(4):
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                outs.append(attend(c, plan(c)))
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert equal(out, refs[i % 2], cs[i % 2]["n"])


def test_pages_far_into_a_large_pool():
    """Pages past 2^31 bytes and 2^31 values into the pool."""
    c = CU.case([140], [1000], seed=20)
    ref = attend(c)
    far = 59000                                             # 4.3e9 bytes, 2.2e9 values
    pool = torch.zeros(far + c["cache"].shape[0], 64, 576, dtype=torch.bfloat16, device="cuda")
    pool[far:] = c["cache"]
    table = torch.where(c["block_table"] < c["cache"].shape[0], c["block_table"] + far, c["block_table"])
    d = dict(c, cache=pool, block_table=table)
    assert equal(attend(d), ref, c["n"])


def test_a_long_context():
    """257 tokens at the end of 40,000 cached rows: scratch past 2^31 bytes; a sample of heads against 64 bits."""
    c = CU.case([257], [40000], seed=21)
    p = plan(c)
    out = attend(c, p)
    assert mla.check(p) == 0
    pick = [0, 1, 77, 127]
    o, _, spread, reach = OC.chunk_attend(c["q"][:, pick], c["w_uk"][pick], c["w_uv"][pick], c["cache"], c["block_table"],
                                          [40000], [0, 257], scale=SCALE)
    off = out[:, pick].double() - o
    assert off.norm() <= 4.4e-3 * o.norm()
    assert (off.abs() <= ((2 * BF * reach + 2e-4 + 2 * BF)[..., None] * spread + BF * o.abs() + 1e-6)).all()


def test_many_requests():
    """More requests than the planner scans at a time, most without tokens (the absorbed form)."""
    rng = np.random.default_rng(22)
    counts = [int(rng.integers(0, 3)) if rng.random() < 0.1 else 0 for _ in range(1500)]
    lens = [int(rng.integers(n, 200)) if n else 0 for n in counts]
    c = CU.case(counts, lens, seed=23)
    p = plan(c)
    out = attend(c, p)
    assert mla.check(p) == 0
    check_absorbed(c, out)


def test_many_prompts():
    """More requests and tiles than the planner scans and ranks at a time; one of the prompts has several tiles."""
    rng = np.random.default_rng(27)
    counts = [int(n) for n in rng.integers(0, 16, 1400)] + [600]
    c = CU.case(counts, [n if n % 3 else n + n // 3 * 30 for n in counts], seed=28, pad=2)
    p = plan(c)
    out = attend(c, p)
    assert mla.check(p) == 0
    pick = [3, 126]
    o, _, spread, reach = OC.chunk_attend(c["q"][:, pick], c["w_uk"][pick], c["w_uv"][pick], c["cache"], c["block_table"],
                                          c["seq_lens"].tolist(), c["offsets"].tolist(), scale=SCALE)
    n = c["n"]
    off, o, spread, reach = (out[:, pick].double() - o)[:n], o[:n], spread[:n], reach[:n]
    assert off.norm() <= 4.4e-3 * o.norm()
    assert (off.abs() <= ((2 * BF * reach + 2e-4 + 2 * BF)[..., None] * spread + BF * o.abs() + 1e-6)).all()


def test_a_prompt_in_chunks_is_the_prompt_at_once():
    c = CU.case([600], [600], seed=24)
    once = attend(c)
    parts = []
    for a, b in ((0, 130), (130, 131), (131, 600)):
        d = dict(c, T=b - a, n=b - a, kv_tokens=-(-b // 64) * 64, q=c["q"][a:b].contiguous(),
                 seq_lens=torch.tensor([b], dtype=torch.int32, device="cuda"),
                 offsets=torch.tensor([0, b - a], dtype=torch.int32, device="cuda"))
        parts.append(attend(d))
    # the same keys, values and weights, in other key tiles: twice a result's own error at most
    off = (torch.cat(parts).double() - once.double()).norm(dim=-1)
    assert (off <= 2 * 1.3e-2 * once.double().norm(dim=-1)).all()


def test_repeated_calls_are_equal_bit_for_bit():
    c = CU.case([700, 129, 5], [3000, 1500, 700], seed=25)
    p = plan(c)
    ref = attend(c, p)
    for _ in range(10):
        assert equal(attend(c, p), ref, c["n"])


def test_refusals():
    c = CU.case([20], [100], seed=26)
    p = plan(c)
    good = dict(scale=SCALE)
    args = [c["q"][..., :128], c["q"][..., 128:], c["w_uk"], c["w_uv"], c["cache"], c["block_table"]]

    def call(i=None, v=None, **kw):
        a = list(args)
        if i is not None:
            a[i] = v
        return mla.chunk_attend(p, *a, **{**good, **kw})

    for i, v in ((0, c["q"][..., :64]), (1, c["q"][:5, :, 128:]), (2, c["w_uk"][:5]), (4, c["cache"][:, :32]), (5, c["block_table"][:, :1]),
                 (0, c["q"][..., 4:132]), (3, c["w_uv"].transpose(1, 2))):
        with pytest.raises(ValueError):
            call(i, v)
    for i, v in ((0, c["q"][..., :128].float()), (5, c["block_table"].long()), (4, CU.quantise(c["cache"]).float())):
        with pytest.raises((TypeError, ValueError)):
            call(i, v)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(mla.MLAError):
            call(scale=scale)
    with pytest.raises(mla.MLAError):
        call(scratch=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        call(scratch=5)
    with pytest.raises(ValueError):
        call(out=torch.empty(20, 128, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        call(lse=torch.empty(20, 64, device="cuda"))
    for kw in (dict(tokens=0), dict(max_pages_per_seq=0), dict(kv_tokens=0), dict(kv_tokens=1 << 31), dict(tokens=1 << 25)):
        with pytest.raises(mla.MLAError):
            mla.chunk_plan(c["seq_lens"], c["offsets"], **{**dict(tokens=20, max_pages_per_seq=2, kv_tokens=128), **kw})
    with pytest.raises(ValueError):
        mla.chunk_plan(c["seq_lens"], c["offsets"][:1], tokens=20, max_pages_per_seq=2)
    with pytest.raises(mla.MLAError):
        mla.chunk_plan(c["seq_lens"], c["offsets"], tokens=20, max_pages_per_seq=2,
                       workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    # a plan's workspace that holds another plan is flagged, and nothing is written
    q = mla.chunk_plan(c["seq_lens"], c["offsets"], tokens=20, max_pages_per_seq=2, kv_tokens=192)
    q.kv_tokens = 128
    out = torch.full((20, 128, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    mla.chunk_attend(q, *args, out=out, **good)
    assert mla.check(q) & mla.MLA_DEV_BAD_PLAN and (out == 7).all()


def test_a_scratch_that_the_memory_does_not_hold(monkeypatch):
    """The call's own scratch: as many heads as a limit or the memory allow, the same bits."""
    import mla_decode_attention_02_gb300._chunk as chunk
    c = CU.case([300, 90], [900, 500], seed=29)
    ref = attend(c)
    asked = []
    real = chunk._attend_in

    def small(*a):
        asked.append(a[10])
        if len(asked) < 4:
            raise torch.OutOfMemoryError("no room")
        return real(*a)

    monkeypatch.setattr(chunk, "_attend_in", small)
    p = plan(c)
    assert equal(attend(c, p), ref, c["n"])
    assert asked == [mla.chunk_scratch_size(p, h) for h in (128, 64, 32, 16)]
    asked.append(0)
    assert equal(attend(c, p), ref, c["n"]) and asked[-1] == asked[3]           # the plan remembers
    monkeypatch.setattr(chunk, "_attend_in", real)
    p = plan(c)
    monkeypatch.setattr(chunk, "CHUNK_SCRATCH_BYTES", mla.chunk_scratch_size(p, 9))
    assert equal(attend(c, p), ref, c["n"]) and p.scratch[False][0] == 8


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_values_beyond_fp16_spoil_what_sees_them_alone(fp8):
    """A later token's row of 1e5 (finite, its values beyond 65504), and weights that hold NaN."""
    c = CU.case([130, 60], [200, 300], seed=30, fp8=fp8)
    ref = attend(c)
    d = CU.case([130, 60], [200, 300], seed=30, fp8=fp8, hold={(0, 150): 1e5})
    d["w_uv"] = d["w_uv"].abs()                            # every value of that row is beyond 1e5
    e = dict(c, w_uv=d["w_uv"])
    ref_abs = attend(e)
    out = attend(d)
    at = 150 - 70                                          # the token of slot 150
    assert equal(out, ref_abs, at) and equal(out[130:], ref_abs[130:], 60)
    assert torch.isnan(out[at:130].float()).all()
    broken = dict(c, w_uv=c["w_uv"].clone())
    broken["w_uv"][3, 5, 7] = float("nan")
    out = attend(broken)
    assert torch.isnan(out[:, 3].float()).all()
    rest = [h for h in range(128) if h != 3]
    assert torch.equal(out[:, rest], ref[:, rest])
