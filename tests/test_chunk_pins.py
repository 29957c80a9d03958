"""The 64-bit oracle of a chunk step pinned to the mathematics, and the C ABI's refusals (no GPU)."""

import cmath
import ctypes
import math

import numpy as np
import pytest
import torch

import chunk_util as CU
import mla_decode_attention_02_gb300 as mla
import mla_decode_attention_02_gb300._chunk as chunk
import oracle.chunk as OC
import oracle.epilog as OE
import oracle.prolog as OP


def test_rates_of_an_unscaled_table():
    r = OC.rates(64)
    assert abs(float(r[0]) - 1) < 1e-15 and abs(float(r[31]) - 10000.0 ** (-62 / 64)) < 1e-18
    assert torch.allclose(r[1:] / r[:-1], torch.full((31,), 10000.0 ** (-2 / 64), dtype=torch.float64), rtol=1e-12)
    assert torch.equal(OC.rates(64, factor=1.0), r)


def test_scaled_rates_keep_fast_pairs_and_slow_the_slow_ones():
    r, s = OC.rates(64), OC.rates(64, factor=40.0)
    turns = 4096 * r / (2 * math.pi)                       # within the original length
    assert torch.equal(s[turns > 32 * 1.5], r[turns > 32 * 1.5])
    assert torch.allclose(s[turns < 1 / 1.5], r[turns < 1 / 1.5] / 40, rtol=1e-12)
    ratio = s / r
    assert (ratio[1:] <= ratio[:-1] + 1e-15).all() and (ratio <= 1).all() and (ratio >= 1 / 40 - 1e-15).all()


@pytest.mark.parametrize("half", [False, True])
def test_rotation_is_complex_multiplication(half):
    x = torch.randn(3, 2, 8, dtype=torch.float64)
    pos, rate = torch.tensor([0, 1, 70000]), OC.rates(8)
    y = OC.rotate(x, pos, rate, half=half)
    for t in range(3):
        for h in range(2):
            for i in range(4):
                a, b = (i, i + 4) if half else (2 * i, 2 * i + 1)
                z = complex(x[t, h, a], x[t, h, b]) * cmath.exp(1j * int(pos[t]) * float(rate[i]))
                assert abs(complex(y[t, h, a], y[t, h, b]) - z) < 1e-9
    assert torch.equal(y[0], x[0])
    back = OC.rotate(y, pos, rate, half=half, inverse=True)
    assert torch.allclose(back, x, atol=1e-12)
    if not half:
        assert np.allclose(OP.rope(x[:, 0].numpy(), pos.numpy(), 10000.0), y[:, 0].numpy(), atol=1e-9)


def test_norm_closed_forms():
    x, w = torch.full((1, 16), 3.0), torch.arange(16.0)
    y, z = OC.residual_norm(x, -x / 3, w, 0.0)
    assert torch.allclose(z, torch.full((1, 16), 2.0, dtype=torch.float64)) and torch.allclose(y[0], w.double())
    y, _ = OC.residual_norm(torch.randn(2, 512), None, torch.ones(512), 0.0)
    assert torch.allclose(y.square().mean(1), torch.ones(2, dtype=torch.float64))
    s, full = OC.group_scales(torch.tensor([[1.0, -4.0] + [0.0] * 126 + [2.0] * 3]).double(), 128)
    assert torch.allclose(s, torch.tensor([[4.0, 2.0]]).double() / 448) and full.shape == (1, 131)
    assert OC.group_scales(torch.zeros(1, 8), 0)[0].item() == 1


def small(counts, lens, **kw):
    c = CU.case(counts, lens, device="cpu", **kw)
    args = (c["q"][:, :2], c["w_uk"][:2], c["w_uv"][:2], c["cache"], c["block_table"], c["seq_lens"].tolist(), c["offsets"].tolist())
    return c, args


def test_attention_is_the_unabsorbed_form_token_by_token():
    c, args = small([3, 0, 4], [3, 0, 68], seed=1, pad=1)
    o, lse, _, _ = OC.chunk_attend(*args, scale=0.07)
    assert torch.isnan(o[7]).all() and torch.isfinite(o[:7]).all()
    for b, t0 in ((0, 0), (2, 3)):
        L, n = int(c["seq_lens"][b]), c["counts"][b]
        rows = OC.cache_rows(c["cache"], c["block_table"][b], L)
        for i in range(n):
            see = rows[:L - n + i + 1]
            want = OE.unabsorbed_attention(c["q"][t0 + i, :2, :128], c["q"][t0 + i, :2, 128:], see[:, :512], see[:, 512:],
                                           c["w_uk"][:2], c["w_uv"][:2], 0.07)
            assert np.allclose(o[t0 + i].numpy(), want, atol=1e-12)


def test_attention_of_one_key_and_of_equal_keys():
    c, args = small([1], [1], seed=2)
    o, lse, _, _ = OC.chunk_attend(*args, scale=0.07)
    v = c["w_uv"][:2].double() @ OC.cache_rows(c["cache"], c["block_table"][0], 1)[0, :512]
    assert torch.allclose(o[0], v)
    c, args = small([2], [50], seed=3)
    c["cache"][int(c["block_table"][0, 0]), :50] = c["cache"][int(c["block_table"][0, 0]), 0].clone()
    o, lse, _, _ = OC.chunk_attend(*args, scale=0.07)
    assert torch.allclose(o[0], o[1], atol=1e-12)
    assert torch.allclose(lse[1] - math.log(50), (c["q"][1, :2].double() * torch.cat(
        [c["w_uk"][:2].double() @ c["cache"][int(c["block_table"][0, 0]), 0, :512].double(),
         c["cache"][int(c["block_table"][0, 0]), 0, 512:].double().expand(2, 64)], 1)).sum(1) * 0.07, atol=1e-9)


def test_what_is_not_seen_counts_nothing_in_the_oracle():
    c, args = small([4], [70], seed=4)
    o, lse, _, _ = OC.chunk_attend(*args, scale=0.07)
    c["cache"][int(c["block_table"][0, 1]), 5] = float("nan")      # slot 69: the last token's
    p, l2, _, _ = OC.chunk_attend(*args, scale=0.07)
    assert torch.equal(p[:3], o[:3]) and torch.isnan(p[3]).all()


def test_fp8_rows_are_the_values_they_stand_for():
    c = CU.case([1], [64], seed=5, device="cpu", fp8=True)
    rows = OC.cache_rows(c["cache"], c["block_table"][0], 64)
    import oracle.fp8 as OF
    assert np.allclose(rows.numpy(), OF.dequantize_cache(c["cache"].numpy())[int(c["block_table"][0, 0])], atol=0)


# ------------------------------------------------------------------------------------ refusals before any CUDA call

A = 0x10000


def test_chunk_calls_refuse_bad_arguments():
    lib = mla.load_library()
    size = ctypes.c_size_t(0)

    def prob(batch=2, tokens=20, heads=128, page=64, pages=4, flags=0, kv=512):
        return ctypes.byref(chunk._Chunk(batch, tokens, heads, page, pages, flags, kv))

    bad = [(dict(batch=0), 1), (dict(tokens=0), 1), (dict(heads=64), 2), (dict(page=32), 2), (dict(pages=0), 1), (dict(flags=1), 1),
           (dict(kv=0), 1), (dict(kv=100), 1), (dict(kv=1 << 30), 2), (dict(tokens=1 << 24), 2), (dict(batch=1 << 25), 2),
           (dict(batch=1 << 10, pages=1 << 22), 2)]
    for kw, want in bad:
        assert lib.mla_chunk_workspace_size(prob(**kw), ctypes.byref(size)) == want, kw
        assert lib.mla_chunk_scratch_size(prob(**kw), 1, 0, ctypes.byref(size)) == want, kw
        assert lib.mla_chunk_plan(prob(**kw), A, A, A, 1 << 20, None) == want, kw
    assert lib.mla_chunk_workspace_size(None, ctypes.byref(size)) == 1
    assert lib.mla_chunk_workspace_size(prob(), None) == 1
    for heads, fp8 in ((0, 0), (129, 0), (1, 2)):
        assert lib.mla_chunk_scratch_size(prob(), heads, fp8, ctypes.byref(size)) == 1
    for args in ((None, A, A), (A, None, A), (A, A, None), (A + 2, A, A), (A, A, A + 8)):
        assert lib.mla_chunk_plan(prob(), *args, 1 << 20, None) == 1

    def attend(fp8=False, **kw):
        a = dict(prob=prob(), qn=A, ns=(24576, 192), qr=A, rs=(24576, 192), uk=A, uv=A, cache=A, pages=8, bt=A, scale=0.07, out=A,
                 lse=A, ws=A, wb=1 << 30, sc=A, sb=1 << 40)
        a.update(kw)
        f = lib.mla_chunk_attend_fp8 if fp8 else lib.mla_chunk_attend
        return f(a["prob"], a["qn"], *a["ns"], a["qr"], *a["rs"], a["uk"], a["uv"], a["cache"], a["pages"], a["bt"], a["scale"],
                 a["out"], a["lse"], a["ws"], a["wb"], a["sc"], a["sb"], None)

    for fp8 in (False, True):
        for k in ("qn", "qr", "uk", "uv", "cache", "bt", "out", "ws", "sc"):
            assert attend(fp8, **{k: None}) == 1, k
        for k, v in (("qn", A + 8), ("out", A + 8), ("bt", A + 2), ("lse", A + 2), ("sc", A + 64), ("ws", A + 8)):
            assert attend(fp8, **{k: v}) == 1, k
        for s in ((0, 192), (24576, 0), (24577, 192), (24576, 12), (1 << 31, 192), (-8, 192)):
            assert attend(fp8, ns=s) == 1 and attend(fp8, rs=s) == 1, s
        for pages in (0, -1, 1 << 31):
            assert attend(fp8, pages=pages) == 1
        for scale in (0.0, -1.0, float("nan"), float("inf")):
            assert attend(fp8, scale=scale) == 1
        assert attend(fp8, prob=None) == 1 and attend(fp8, prob=prob(heads=1)) == 2


def test_rotation_and_norm_refuse_bad_arguments():
    lib = mla.load_library()

    def rotate(tokens=4, heads=8, dims=64, x=A, xs=(512, 64), pos=A, table=A, layout=0, inverse=0, m=1.0, out=2 * A, os=(512, 64)):
        return lib.mla_rotate(tokens, heads, dims, x, *xs, pos, table, layout, inverse, m, out, *os, None)

    for kw in (dict(tokens=0), dict(heads=0), dict(layout=2), dict(inverse=2), dict(m=float("nan")), dict(m=float("inf")), dict(x=None),
               dict(out=None), dict(pos=None), dict(table=None), dict(x=A + 8), dict(pos=A + 1), dict(xs=(0, 64)), dict(xs=(512, 4)),
               dict(os=(512, -8)), dict(os=(1 << 31, 64)), dict(out=A, os=(1024, 64))):
        assert rotate(**kw) == 1, kw
    for kw in (dict(dims=48), dict(dims=512), dict(dims=8), dict(tokens=1 << 24, heads=1 << 8)):
        assert rotate(**kw) == 2, kw
    nan, inf = float("nan"), float("inf")
    for args in ((1.0, 64, 2.0, 4096, 32.0, 1.0), (nan, 64, 2.0, 4096, 32.0, 1.0), (1e4, 48, 2.0, 4096, 32.0, 1.0),
                 (1e4, 64, 0.5, 4096, 32.0, 1.0), (1e4, 64, inf, 4096, 32.0, 1.0), (1e4, 64, 2.0, 0, 32.0, 1.0),
                 (1e4, 64, 2.0, 4096, 0.5, 1.0), (1e4, 64, 2.0, 4096, 32.0, 0.0), (1e4, 64, 2.0, 4096, inf, 1.0)):
        assert lib.mla_rope_table_scaled(*args, A, None) == 1, args
    assert lib.mla_rope_table_scaled(1e4, 64, 2.0, 4096, 32.0, 1.0, None, None) == 1

    def norm(tokens=4, hidden=64, x=A, xs=64, r=A, rs=64, w=A, eps=1e-6, out=A, kept=A, group=None, scales=A):
        if group is None:
            return lib.mla_residual_norm(tokens, hidden, x, xs, r, rs, w, eps, out, kept, None)
        return lib.mla_residual_norm_fp8(tokens, hidden, x, xs, r, rs, w, eps, group, out, scales, kept, None)

    for group in (None, 0, 128):
        for kw in (dict(tokens=0), dict(hidden=0), dict(x=None), dict(w=None), dict(out=None), dict(x=A + 8), dict(r=A + 8), dict(kept=A + 8),
                   dict(xs=0), dict(xs=12), dict(rs=-8), dict(xs=1 << 31), dict(eps=-1.0), dict(eps=nan), dict(eps=inf)):
            assert norm(group=group, **kw) == 1, kw
        for kw in (dict(hidden=12), dict(hidden=16392)):
            assert norm(group=group, **kw) == 2, kw
    assert norm(group=64) == 2 and norm(group=-1) == 2 and norm(group=128, scales=None) == 1 and norm(group=0, scales=A + 2) == 1
    assert norm(group=128, out=A + 4) == 1


def test_the_binding_refuses_what_is_not_on_a_gpu():
    cpu = torch.zeros(4, 128, 192, dtype=torch.bfloat16)
    lens = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: mla.rotate(cpu[..., 128:], lens, table=None), lambda: mla.residual_norm(cpu[0], None, None),
                 lambda: mla.residual_norm_fp8(cpu[0], None, None),
                 lambda: mla.chunk_plan(lens, lens, tokens=4, max_pages_per_seq=1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        mla.residual_norm([1.0], None, None)
