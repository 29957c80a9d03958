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
    o, l, _, _ = OC.chunk_attend(c["q"], c["w_uk"], c["w_uv"], c["cache"], c["block_table"], c["seq_lens"].tolist(),
                                 c["offsets"].tolist(), scale=SCALE)
    n = c["n"]
    off, size = (out[:n].double() - o[:n]).norm(dim=-1), o[:n].norm(dim=-1)
    assert off.norm() <= 6e-3 * size.norm() and (off <= 1.8e-2 * size).all(), (off.norm() / size.norm(), (off / size).max())
    # sum |q_latent c| over 512 products of a normal q_latent of size 1 / sqrt(2) ... 0.82 and a normal c: below 512
    assert (lse[:n].double() - l[:n]).abs().max() <= BF * SCALE * 512
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
