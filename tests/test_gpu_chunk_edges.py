"""Chunk attention where its roundings and its choice of form could show: against 64 bits, with keys that are exact.

W_UK picks a latent value for each key dimension (``exact_keys``), so a key is a cached bf16 value and no key is rounded.
Half a step is BF = 2^-8 of the value in bf16, FP = 2^-11 in fp16.  What is left in the form with per-head keys:

* a score: 192 products summed in fp32, off by 192 2^-23 of scale sum |q k| at most; its product with log2(e) and the shift by the
  reference, 2^-22 of it: d = 24e-6 * reach.
* weights rounded once and values rounded once, FP each (and 1e-6 for the exponential), the output once, BF:
  |o - ref| <= (exp(2 d) - 1 + 2 FP + 1e-6) spread + BF |ref|, and |lse - ref| <= d + 1e-5.
* a value itself is a sum of 512 products in fp32: 512 2^-24 sum |w r| more at most, and where it is below fp16's normal values
  2^-25 more: both absolute, and weighted averages of them over the keys are no larger than the largest.  (Small beside the
  other terms but where one key has all the weight and its value is next to nothing.)
* in the mean square BF / sqrt(3) = 2.26e-3 and twice FP / sqrt(3) = 2.8e-4 of o's norm: 2.3e-3; a row three times that.
  (bf16 weights and values, three roundings of 1.66e-3 as they come out, would make 2.9e-3.)
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
BF, FP = 2.0 ** -8, 2.0 ** -11
HEADS = [0, 1, 77, 127]


def plan(c, **kw):
    kw.setdefault("kv_tokens", c["kv_tokens"])
    return mla.chunk_plan(c["seq_lens"], c["offsets"], tokens=c["T"], max_pages_per_seq=c["block_table"].shape[1], **kw)


def attend(c, p=None, **kw):
    f = mla.chunk_attend_fp8 if c["cache"].dtype == torch.uint8 else mla.chunk_attend
    return f(p or plan(c), c["q"][..., :128], c["q"][..., 128:], c["w_uk"], c["w_uv"], c["cache"], c["block_table"],
             scale=SCALE, **kw)


def exact_keys(c):
    """Key dimension d of head h is latent value (d + 4 h) mod 512."""
    h, d = torch.arange(128, device="cuda")[:, None], torch.arange(128, device="cuda")[None, :]
    c["w_uk"] = torch.zeros_like(c["w_uk"])
    c["w_uk"][h, d, (d + 4 * h) % 512] = 1
    return c


def oracle(c, heads):
    o, lse, spread, _ = OC.chunk_attend(c["q"][:, heads], c["w_uk"][heads], c["w_uv"][heads], c["cache"], c["block_table"],
                                        c["seq_lens"].tolist(), c["offsets"].tolist(), scale=SCALE)
    return o, lse, spread


def reach_of(c, heads):
    """[T][heads] largest scale * sum |q k| over all 192 dimensions of the keys seen (an upper bound: over all keys)."""
    out = torch.zeros(c["T"], len(heads), dtype=torch.float64, device="cuda")
    off = c["offsets"].tolist()
    for b, L in enumerate(c["seq_lens"].tolist()):
        t = slice(off[b], off[b + 1])
        if off[b] == off[b + 1]:
            continue
        rows = OC.cache_rows(c["cache"], c["block_table"][b], L)
        for i, h in enumerate(heads):
            k = torch.cat([rows[:, :512] @ c["w_uk"][h].double().T, rows[:, 512:]], 1).abs()
            out[t, i] = SCALE * (c["q"][t, h].double().abs() @ k.T).amax(1)
    return out


def value_sums(c, heads):
    """[heads][128] largest sum |w r| of a value over the keys of all requests."""
    rows = torch.cat([OC.cache_rows(c["cache"], c["block_table"][b], L)
                      for b, (L, n) in enumerate(zip(c["seq_lens"].tolist(), c["counts"])) if n])
    return torch.stack([(rows[:, :512].abs() @ c["w_uv"][h].double().abs().T).amax(0) for h in heads])


def check_exact(c, out, lse, heads=HEADS):
    o, l, spread = oracle(c, heads)
    n, d = c["n"], 24e-6 * reach_of(c, heads)
    o, l, spread, d, got = o[:n], l[:n], spread[:n], d[:n], out[:n, heads].double()
    value = 512 * 2.0 ** -24 * value_sums(c, heads) + 2.0 ** -25
    bound = (torch.exp(2 * d) - 1 + 2 * FP + 1e-6)[..., None] * spread + BF * o.abs() + value
    assert ((got - o).abs() <= bound).all(), ((got - o).abs() - bound).max()
    assert ((lse[:n, heads].double() - l).abs() <= d + 1e-5).all()
    return o, got, bound


@pytest.mark.parametrize("gap", [8.0, 14.0, 16.0, 17.5])
@pytest.mark.parametrize("tokens", [120, 200], ids=["halves", "tiles"])
def test_a_first_key_that_draws_nearly_all_the_weight(tokens, gap):
    """A sink: key 0 stands `gap` (in natural units) above the others' mean and its value is zero, so the output is what
    the 32767 small weights make; at 17.5 they are 2^-25 of it each, 1.4e-3 of the weight in all.

    fp16's steps end at 2^-24 (half of one: 2^-25, 2^-25 / sqrt(3) in the mean square).  The weights stand at least 2^7 above the
    largest, and where 64 of them in a row are below 2^-20 of it the reference falls to theirs: so the others' mean square is
    2^-16 or more (20 log2 units below 2^7, and 3.5 of the largest of 64 above the mean), their error 2^-9.8 of it at most: 1.1e-3
    beside the 2.3e-3, 2.5e-3 in all.  The 63 keys of the first half tile stay where they are: 4% of the norm, off by 2^-6 of theirs.
    """
    L = 32768
    c = exact_keys(CU.case([tokens], [L], seed=61, poison=False))
    first = int(c["block_table"][0, 0])
    c["cache"][first, 0, :575] = 0
    c["cache"][:, :, 575] = 0
    c["q"][..., 191] = 16
    c["cache"][first, 0, 575] = gap / (16 * SCALE)
    lse = torch.empty(tokens, 128, device="cuda")
    p = plan(c)
    out = attend(c, p, lse=lse)
    assert mla.check(p) == 0
    o, l, _ = oracle(c, HEADS)
    off, size = (out[:, HEADS].double() - o).norm(dim=-1), o.norm(dim=-1)
    assert off.norm() <= 2.5e-3 * size.norm() and (off <= 7e-3 * size).all(), (off.norm() / size.norm(), (off / size).max())
    assert (lse[:, HEADS].double() - l).abs().max() <= 1e-3


@pytest.mark.parametrize("scale", [1.0, 4.0, 30.0])
def test_rising_scores_to_a_rounding(scale):
    """Keys that grow along the context, so that the reference is raised again and again and the outputs rescaled."""
    lens = [900, 700]
    c = exact_keys(CU.case([200, 60], lens, seed=62))
    c["q"] *= scale
    grow = torch.linspace(0.2, 3.0, 960, device="cuda").to(torch.bfloat16)
    for b, L in enumerate(lens):
        for j in range(-(-L // 64)):
            c["cache"][int(c["block_table"][b, j])] *= grow[j * 64:j * 64 + 64][:, None]
    lse = torch.empty(c["T"], 128, device="cuda")
    out = attend(c, lse=lse)
    o, got, bound = check_exact(c, out, lse)
    for wrong in (torch.zeros_like(o), 0.5 * o, 1.05 * o):                   # (what the bound has to tell from the output)
        assert ((wrong - o).abs() > bound).float().mean() > 0.5


@pytest.mark.parametrize("counts,lens", [([700], [700]), ([100, 0, 300, 128], [700, 0, 301, 400]), ([257], [1000]), ([1], [1])],
                         ids=["prompt", "ragged", "tiles", "one"])
def test_weights_and_values_have_sixteen_bit_steps_of_fp16(counts, lens):
    c = exact_keys(CU.case(counts, lens, seed=63))
    lse = torch.empty(c["T"], 128, device="cuda")
    out = attend(c, lse=lse)
    o, got, _ = check_exact(c, out, lse)
    off, size = (got - o).norm(dim=-1), o.norm(dim=-1)
    assert off.norm() <= 2.3e-3 * size.norm() and (off <= 6.9e-3 * size).all(), (off.norm() / size.norm(), (off / size).max())


@pytest.mark.parametrize("scale", [1.0, 6.0])
def test_scores_that_go_up_and_down(scale):
    """A reference that is raised and falls in turn: blocks of 1024 keys whose scores lie far apart, in no order."""
    c = exact_keys(CU.case([140, 100], [9000, 5000], seed=64, poison=False))
    c["q"][..., 191] = 8
    steps = torch.tensor([0.0, 12.0, -20.0, -45.0, 14.0, -30.0, -6.0, 3.0, -60.0], device="cuda") / (8 * SCALE)
    for b, L in enumerate((9000, 5000)):
        for j in range(-(-L // 64)):
            c["cache"][int(c["block_table"][b, j]), :, 575] = float(steps[j // 16 % 9])
    c["q"][..., :191] *= scale
    lse = torch.empty(c["T"], 128, device="cuda")
    check_exact(c, attend(c, lse=lse), lse)


def test_scores_that_fall_without_end():
    """25 log2 units down every 512 keys: what is far below counts nothing, and nothing passes fp32's range."""
    c = exact_keys(CU.case([130], [12000], seed=65, poison=False))
    c["q"][..., 191] = 16
    for j in range(188):
        c["cache"][int(c["block_table"][0, j]), :, 575] = -17.0 * (j // 8) / (16 * SCALE)
    lse = torch.empty(c["T"], 128, device="cuda")
    check_exact(c, attend(c, lse=lse), lse)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("field,value", [("tokens", 22), ("max_pages", 46), ("batch", 2)])
def test_another_plan_in_the_workspace_of_few_tokens(field, value, fp8):
    """The absorbed form, as the other: what the plan in the workspace is not for is flagged, and nothing is written."""
    c = CU.case([3, 0, 20], [3000, 0, 2500], seed=66, fp8=fp8, spare=0)
    p = plan(c)
    setattr(p, field, value)
    d = dict(c, q=c["q"][:p.tokens], block_table=c["block_table"][:p.batch, :p.max_pages].contiguous())
    out = torch.full((p.tokens, 128, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.tokens, 128), 7.0, device="cuda")
    attend(d, p, out=out, lse=lse)
    assert mla.check(p) & mla.MLA_DEV_BAD_PLAN
    assert (out == 7).all() and (lse == 7).all()
