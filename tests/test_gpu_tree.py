"""GPU parity of the tree step (query, cache append, tree attention, commit) with the fp64 oracle.

Tolerances, from the roundings (bf16: half a step is at most 2^-8 of the value):

* tree attention: a weight is rounded to bf16 once, and again if its page half is rescaled to the pair's
  maximum; o is rounded once; a score's fp32 error is below 576 2^-24 scale sum|q k| < 1.2e-3 for these N(0, 1)
  inputs (sum|q k| has mean 367 and deviation 15: 480 is far out), which moves a weight by twice that at most
  (through its own score and through the sum) and lse by once.
  So |o - ref| <= (2 2^-8 + 2.4e-3) sum_j w_j |v_j| + 2^-8 |ref| + 1e-6 and |lse - ref| <= 1.2e-3.
* query: one bf16 rounding, 128 fp32 products and sums (128 2^-24 sum|q w|); the rotation's angle is good to
  1e-5 rad and the sine and cosine to 1e-6, both times the pair's size.
* append: one bf16 rounding after fp32 arithmetic of a few steps (1e-5 relative); fp8 codes half an e4m3 step
  (2^-4 of the value, 2^-10 below the normal range, in units of the row's scale).
"""

import numpy as np
import pytest
import torch

import mla_decode_attention_02_gb300 as mla
import oracle.fp8 as OF
import oracle.prolog as OP
import oracle.tree as OT
import tree_util as TU

pytestmark = pytest.mark.gpu
SCALE = mla.DEFAULT_SCALE
BF = 2.0 ** -8


def f64(t):
    return t.detach().double().cpu().numpy()


def run_tree(c, ql, qr, cache, fp8=False, max_pages=None, **kw):
    d = TU.index_tensors(c)
    p = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=d["block_table"].shape[1])
    out = torch.full((c["T"], 128, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c["T"], 128), 7.0, dtype=torch.float32, device="cuda")
    f = mla.tree_decode_fp8 if fp8 else mla.tree_decode
    f(p, ql.cuda(), qr.cuda(), cache.cuda(), d["block_table"], scale=SCALE, out=out, lse=lse, **kw)
    return out, lse, mla.check(p), p


def check_rows(out, lse, ref, rows, what=""):
    o, l, spread = ref
    got, got_l = f64(out)[rows], f64(lse)[rows]
    o, l, spread = o[rows], l[rows], spread[rows]
    assert np.isfinite(got).all(), what
    over = np.abs(got - o) - ((2 * BF + 2.4e-3) * spread + BF * np.abs(o) + 1e-6)
    assert over.max() <= 0, f"{what}: o beyond its bound by {over.max():.3e}"
    inf = np.isinf(l)
    assert np.array_equal(np.isneginf(got_l), inf), what
    assert np.abs(got_l[~inf] - l[~inf]).max(initial=0) <= 1.2e-3, what


def fp8_of(cache):
    """fp8 rows of a bf16 cache; rows that hold NaN become NaN codes and a NaN scale."""
    bad = torch.isnan(cache.float()).any(-1)
    rows = torch.from_numpy(OF.quantize_cache(torch.where(bad[..., None], torch.zeros((), dtype=cache.dtype), cache)))
    rows[bad] = 0x7F
    return rows


CASES = [
    # counts, lens, masks
    ([1], [1], "tree"),                                   # one node, no context
    ([1], [2], "tree"),
    ([1, 1, 1], [63, 64, 65], "tree"),
    ([64], [64], "tree"),                                 # a tree alone, one page
    ([64], [65], "bits"),                                 # one key of context, the tree over two pages
    ([64, 33], [127, 128], "bits"),
    ([7, 5, 16, 3], [40, 700, 129, 3], ["tree", "bits", "self", "chain"]),
    ([5, 0, 9, 0], [200, 0, 75, 10 ** 9], "tree"),        # slots of the batch without a request
    ([3, 4], [3, 68], "none"),                            # nodes that see no key; nodes that see the context alone
    ([8, 8], [8, 90], ["bits", "all"]),
    ([2], [6000], "chain"),                               # rows cut into pieces over the units
    ([40, 1], [1500, 3001], "tree"),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("counts,lens,kind", CASES, ids=[f"{i}" for i in range(len(CASES))])
def test_tree_decode_parity(counts, lens, kind, fp8):
    c = TU.case(counts, lens, kind, seed=11, pad=2)
    ql, qr, cache = TU.tensors(c, seed=12)
    if fp8:
        cache = fp8_of(cache)
        ref_cache = np.nan_to_num(OF.dequantize_cache(cache.numpy()), nan=np.nan)
    else:
        ref_cache = cache
    ref = OT.tree_decode(ql, qr, ref_cache, c["block_table"], c["seq_lens"], c["offsets"], c["masks"], scale=SCALE)
    out, lse, status, p = run_tree(c, ql, qr, cache, fp8)
    assert status == 0
    n = int(c["offsets"][-1])
    check_rows(out, lse, ref, slice(0, n))
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()          # rows behind the last request
    empty = np.isneginf(ref[1][:n])
    assert (f64(out)[:n][empty] == 0).all()


def test_tree_fp8_scratch_changes_no_bit():
    c = TU.case([7, 0, 64, 16, 3], [40, 9, 700, 129, 3], ["tree", "tree", "bits", "self", "chain"], seed=13, pad=2)
    ql, qr, cache = TU.tensors(c, seed=14)
    cache = fp8_of(cache)
    out, lse, status, p = run_tree(c, ql, qr, cache, True, scratch=False)
    n = len(c["counts"]) * c["block_table"].shape[1] * mla.EXPANDED_PAGE_BYTES
    room = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")       # NaN in whatever is not expanded
    for s in (room, None):
        o2, l2, st2, _ = run_tree(c, ql, qr, cache, True, scratch=s)
        assert status == st2 == 0
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    a = run_tree(c, ql, qr, cache, True, scratch=False, pow2_max=False)
    b = run_tree(c, ql, qr, cache, True, scratch=room, pow2_max=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ref = OT.tree_decode(ql, qr, OF.dequantize_cache(cache.numpy()), c["block_table"], c["seq_lens"], c["offsets"],
                         c["masks"], scale=SCALE)
    check_rows(a[0], a[1], ref, slice(0, int(c["offsets"][-1])))
    c["block_table"][3, 1] = c["pages"]                                  # a bad page: the same rows, the same flag
    a = run_tree(c, ql, qr, cache, True, scratch=False)
    b = run_tree(c, ql, qr, cache, True, scratch=room)
    assert a[2] == b[2] == mla.MLA_DEV_BAD_PAGE
    assert torch.equal(torch.nan_to_num(a[0], nan=9.0), torch.nan_to_num(b[0], nan=9.0))
    with pytest.raises(mla.MLAError, match="workspace"):
        run_tree(c, ql, qr, cache, True, scratch=room[:-16])


def test_tree_decode_pow2():
    c = TU.case([9, 12], [300, 2000], "tree", seed=21)
    ql, qr, cache = TU.tensors(c, seed=22)
    ref = OT.tree_decode(ql, qr, cache, c["block_table"], c["seq_lens"], c["offsets"], c["masks"], scale=SCALE)
    out, lse, status, _ = run_tree(c, ql, qr, cache, pow2_max=True)
    assert status == 0
    check_rows(out, lse, ref, slice(None))


def test_tree_infinite_and_huge_values_in_masked_rows():
    c = TU.case([6, 20], [100, 500], "self", seed=23)
    ql, qr, cache = TU.tensors(c, seed=24)
    # node 3 of the first tree is seen by itself alone: its row spoils no other node
    L, n = 100, 6
    slot = L - n + 3
    page = int(c["block_table"][0][slot // 64])
    clean = cache.clone()
    ref = OT.tree_decode(ql, qr, clean, c["block_table"], c["seq_lens"], c["offsets"], c["masks"], scale=SCALE)
    others = [t for t in range(26) if t != 3]
    for value in (float("inf"), float("-inf"), float("nan"), 3e38):
        cache[page, slot % 64] = value
        out, lse, status, _ = run_tree(c, ql, qr, cache)
        assert status == 0
        check_rows(out[others], lse[others], tuple(x[others] for x in ref), slice(None), str(value))


def test_tree_of_a_chain_is_the_two_token_decode():
    c = TU.case([2] * 5, [2, 65, 700, 4000, 129], "chain", seed=25)
    ql, qr, cache = TU.tensors(c, seed=26)
    out, lse, status, _ = run_tree(c, ql, qr, cache)
    d = TU.index_tensors(c)
    table = torch.where(d["block_table"] == 1 << 30, -1, d["block_table"])
    p = mla.plan(d["seq_lens"], s_q=2, max_pages_per_seq=table.shape[1])
    o2, l2 = mla.decode(p, ql.cuda().view(5, 2, 128, 512), qr.cuda().view(5, 2, 128, 64), cache.cuda(), table, scale=SCALE)
    assert status == 0 and mla.check(p) == 0
    # the same kernel on other cuts of the rows: each side within its own bound of the formula
    ref = OT.tree_decode(ql, qr, cache, c["block_table"], c["seq_lens"], c["offsets"], c["masks"], scale=SCALE)
    check_rows(out, lse, ref, slice(None))
    check_rows(o2.view(10, 128, 512), l2.view(10, 128), ref, slice(None))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_tree_batch_without_requests(fp8):
    c = TU.case([0, 0, 0], [0, 7, -3], "tree", seed=29, pad=5, width=2)
    ql, qr, cache = TU.tensors(c, seed=30)
    out, lse, status, _ = run_tree(c, ql, qr, fp8_of(cache) if fp8 else cache, fp8)
    assert status == 0 and (out == 7).all() and (lse == 7).all()


def test_tree_bad_inputs_are_flagged():
    c = TU.case([4, 4, 4], [100, 3, 300], "tree", seed=27, pad=1)
    ql, qr, cache = TU.tensors(c, seed=28)
    ref = OT.tree_decode(ql[:4], qr[:4], cache, c["block_table"][:1], c["seq_lens"][:1], c["offsets"][:2], c["masks"],
                         scale=SCALE)
    c["block_table"][2, 1] = c["pages"]                      # outside the pool
    out, lse, status, _ = run_tree(c, ql, qr, cache)
    assert status == mla.MLA_DEV_BAD_SEQ_LEN | mla.MLA_DEV_BAD_PAGE
    check_rows(out, lse, ref, slice(0, 4))
    assert torch.isnan(out[4:12]).all() and torch.isnan(lse[4:12]).all()
    assert (out[12:] == 7).all()
    c["offsets"][1] = 9                                      # decreasing
    out, lse, status, _ = run_tree(c, ql, qr, cache)
    assert status == mla.MLA_DEV_BAD_OFFSETS and torch.isnan(out).all() and torch.isnan(lse).all()


def test_tree_plan_matches_the_host():
    for seed, (counts, lens) in enumerate([([7, 0, 64, 1], [900, 5, 64, 9000]), ([16] * 30, list(range(20, 3020, 100))),
                                           ([3], [3]), ([2] * 9, [70] * 9), ([64] * 31 + [1, 17], [64 + 5 * i for i in range(33)]),
                                           ([8], [700]), ([1, 0, 3], [8192, 1, 2500]), ([12, 12], [40000, 39000]),
                                           ([33] * 300, [33 + i % 900 for i in range(300)])]):
        c = TU.case(counts, lens, "tree", seed=seed, pad=seed)
        d = TU.index_tensors(c)
        p = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=c["block_table"].shape[1])
        got = mla.tree_plan_device(p)
        want = mla.tree_plan_host(c["seq_lens"], c["offsets"], c["masks"], max_pages_per_seq=c["block_table"].shape[1],
                                  num_units=mla.num_units())
        assert got["header"] == want["header"]
        n = int(c["offsets"][-1])
        for k in ("items", "item_unit", "unit_begin", "row_nparts", "row_part0", "row_item0", "tree_pages", "tree_items"):
            assert np.array_equal(got[k], want[k]), k
        assert np.array_equal(got["tree_rows"][:n], want["tree_rows"][:n])


def test_tree_many_rows_and_repeats():
    """More rows than units, the same bits every time, in a captured graph and on another stream too."""
    c = TU.case([11] * 30, [int(x) for x in np.linspace(11, 1400, 30)], "tree", seed=31)
    ql, qr, cache = TU.tensors(c, seed=32)
    ref = OT.tree_decode(ql, qr, cache, c["block_table"], c["seq_lens"], c["offsets"], c["masks"], scale=SCALE)
    out, lse, status, p = run_tree(c, ql, qr, cache)
    assert status == 0
    check_rows(out, lse, ref, slice(None))
    d = TU.index_tensors(c)
    qlc, qrc, kv = ql.cuda(), qr.cuda(), cache.cuda()
    for _ in range(5):
        o2, l2 = mla.tree_decode(p, qlc, qrc, kv, d["block_table"], scale=SCALE)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p2 = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=c["block_table"].shape[1], stream=s)
    o2, l2 = mla.tree_decode(p2, qlc, qrc, kv, d["block_table"], scale=SCALE, stream=s)
    s.synchronize()
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    og, lg = torch.zeros_like(out), torch.zeros_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p3 = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=c["block_table"].shape[1])
        mla.tree_decode(p3, qlc, qrc, kv, d["block_table"], scale=SCALE, out=og, lse=lg)
    for _ in range(2):
        og.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(og, out) and torch.equal(lg, lse)


def test_trees_on_two_streams_at_once():
    cases = [TU.case([9, 30, 5], [1500, 700, 3000], "tree", seed=71), TU.case([16] * 6, [900] * 6, "bits", seed=72)]
    data = [TU.tensors(c, seed=73 + i) for i, c in enumerate(cases)]
    alone = [run_tree(c, *t)[:2] for c, t in zip(cases, data)]
    dev = [(TU.index_tensors(c), [x.cuda() for x in t]) for c, t in zip(cases, data)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(6):
        for i, (d, t) in enumerate(dev):
            p = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=d["block_table"].shape[1],
                              stream=streams[i])
            got[i].append(mla.tree_decode(p, *t, d["block_table"], scale=SCALE, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for o, l in got[i]:
            assert torch.equal(o, alone[i][0]) and torch.equal(l, alone[i][1])


def test_rows_past_32_bit_offsets():
    """A pool whose last pages lie past 2^31 elements: append, attention and commit there."""
    pages = 60000                                                 # 2.2e9 elements, 4.4 GB
    pool = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    c = TU.case([5, 3], [70, 131], "tree", seed=75, spare=0)
    c["block_table"] = np.where(c["block_table"] < 1 << 30, pages - 1 - c["block_table"], -1).astype(np.int32)
    d = TU.index_tensors(c)
    g = torch.Generator().manual_seed(76)
    kv = torch.randn(201, 576, generator=g).to(torch.bfloat16).cuda()
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    st = mla.cache_append(kv[:, :512], kv[:, 512:], gamma, pool, d["block_table"], d["seq_lens"],
                          torch.tensor([0, 70, 201], dtype=torch.int32, device="cuda"))
    assert st.item() == 0
    used = pool[pages - 8:].cpu()
    small = TU.case([5, 3], [70, 131], "tree", seed=75, spare=0)
    table = np.where(c["block_table"] >= 0, c["block_table"] - (pages - 8), 0)
    slots = OT.token_slots(table, c["seq_lens"], [0, 70, 201])
    lat, rope = OT.token_rows(f64(kv)[:, :512], f64(kv)[:, 512:], np.ones(512), [s for _, _, s in slots])
    rows = f64(used.reshape(-1, 576))
    at = [r for _, r, _ in slots]
    assert (np.abs(rows[at][:, :512] - lat) <= (BF + 1e-5) * np.abs(lat)).all()
    ql, qr, _ = TU.tensors(small, seed=77)
    p = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=d["block_table"].shape[1])
    o, lse = mla.tree_decode(p, ql.cuda(), qr.cuda(), pool, d["block_table"], scale=SCALE)
    assert mla.check(p) == 0
    ref = OT.tree_decode(ql, qr, used, table, c["seq_lens"], c["offsets"], c["masks"], scale=SCALE)
    check_rows(o, lse, ref, slice(None))
    paths = np.array([[0, 3, 4], [1, 2, 0]], np.int32)
    plens = np.array([3, 2], np.int32)
    new, st = mla.cache_commit(pool, d["block_table"], d["seq_lens"], d["offsets"], torch.from_numpy(paths).cuda(),
                               torch.from_numpy(plens).cuda())
    want, lens = OT.commit(used.view(torch.int16).reshape(-1, 576).numpy(), table, c["seq_lens"], c["offsets"], paths, plens)
    assert st.item() == 0 and new.cpu().tolist() == lens.tolist()
    assert np.array_equal(pool[pages - 8:].cpu().view(torch.int16).reshape(-1, 576).numpy(), want)
    assert not pool[:pages - 8].any()


def test_query_past_32_bit_offsets():
    T = 33000                                                     # 2.16e9 output values
    g = torch.Generator(device="cuda").manual_seed(78)
    q = torch.randn(T, 128, 192, generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(128, 128, 512, generator=g, device="cuda", dtype=torch.bfloat16) * 128 ** -0.5
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    ql, qr, st = mla.query(q[..., :128], q[..., 128:], w, pos)
    assert st.item() == 0
    for at in (0, T - 60):                                         # a small call's rows are the same
        a, b, _ = mla.query(q[at:at + 60, :, :128], q[at:at + 60, :, 128:], w, pos[at:at + 60])
        assert torch.equal(ql[at:at + 60], a) and torch.equal(qr[at:at + 60], b)


def test_tree_refuses_wrong_arguments():
    c = TU.case([3], [100], "tree", seed=33)
    ql, qr, cache = TU.tensors(c, seed=34)
    d = TU.index_tensors(c)
    p = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=2)
    ql, qr, cache = ql.cuda(), qr.cuda(), cache.cuda()
    with pytest.raises(ValueError, match="q_latent"):
        mla.tree_decode(p, ql[:2], qr, cache, d["block_table"])
    with pytest.raises(TypeError, match="kv_cache"):
        mla.tree_decode_fp8(p, ql, qr, cache, d["block_table"])
    with pytest.raises(ValueError, match="block_table"):
        mla.tree_decode(p, ql, qr, cache, d["block_table"][:, :1])
    with pytest.raises(mla.MLAError):
        mla.tree_decode(p, ql, qr, cache, d["block_table"], scale=-1.0)
    with pytest.raises(ValueError, match="token_offsets"):
        mla.tree_plan(d["seq_lens"], d["offsets"][:1], d["masks"], max_pages_per_seq=2)
    with pytest.raises(mla.MLAError):
        mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=2,
                      workspace=torch.empty(4096, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="scratch"):
        mla.tree_decode_fp8(p, ql, qr, torch.zeros(9, 64, 656, dtype=torch.uint8, device="cuda"), d["block_table"],
                            scratch=True)
    big = torch.zeros(20000, dtype=torch.int64, device="cuda")
    with pytest.raises(mla.MLAError, match="unsupported"):
        mla.tree_plan(d["seq_lens"], d["offsets"], big, max_pages_per_seq=2)


# ---------------------------------------------------------------- query

@pytest.mark.parametrize("T", [1, 7, 127, 128, 129, 300])
@pytest.mark.parametrize("strided", [False, True], ids=["dense", "views"])
def test_query_parity(T, strided):
    g = torch.Generator().manual_seed(T)
    q = torch.randn(T, 128, 192, generator=g).to(torch.bfloat16)
    w = (torch.randn(128, 128, 512, generator=g) * 128 ** -0.5).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    pos[0] = 0
    if T > 3:
        pos[1], pos[2], pos[3] = (1 << 20) - 1, -1, -7          # the farthest; two tokens left out
    qc = q.cuda()
    qn, qp = (qc[..., :128], qc[..., 128:]) if strided else (qc[..., :128].contiguous(), qc[..., 128:].contiguous())
    ql = torch.full((T, 128, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    qr = torch.full((T, 128, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    _, _, st = mla.query(qn, qp, w.cuda(), pos.cuda(), q_latent=ql, q_rope=qr)
    assert st.item() == 0
    keep = pos.numpy() >= 0
    assert (ql.cpu()[~torch.from_numpy(keep)] == 7).all() and (qr.cpu()[~torch.from_numpy(keep)] == 7).all()
    x, wd = f64(q), f64(w)
    ref = OP.absorb_q(x[keep][..., :128], wd)
    size = OP.absorb_q(np.abs(x[keep][..., :128]), np.abs(wd))
    got = f64(ql)[keep]
    assert (np.abs(got - ref) <= BF * np.abs(ref) + 128 * 2.0 ** -24 * size + 1e-30).all()
    ref = OP.rope(x[keep][..., 128:], pos.numpy()[keep][:, None], 10000.0)
    pe = x[keep][..., 128:].reshape(-1, 128, 32, 2)
    pair = np.repeat(np.abs(pe).sum(-1), 2, axis=-1)
    assert (np.abs(f64(qr)[keep] - ref) <= BF * np.abs(ref) + 2e-5 * pair).all()


@pytest.mark.parametrize("B", [3, 100], ids=["few", "many"])
def test_query_equals_the_prolog(B):
    import workloads as W
    t = W.prolog_tensors(B, 2, 5)
    c = W.sparse_cache([700, 64, 9000][:B] + [65 + 31 * i for i in range(B - 3)], 2, 5)
    d = {k: v.cuda() for k, v in t.items() if isinstance(v, torch.Tensor)}
    ql, qr, _ = mla.prolog(d["q_nope"], d["q_pe"], d["kv_latent"], d["k_pe"], d["w_uk"], d["kv_norm_weight"],
                           c["kv_cache"].cuda(), c["block_table"].cuda(), c["seq_lens"].cuda())
    pos = (c["seq_lens"][:, None] - 2 + torch.arange(2)).to(torch.int32).view(-1).cuda()
    a, b, _ = mla.query(d["q_nope"].view(2 * B, 128, 128), d["q_pe"].view(2 * B, 128, 64), d["w_uk"], pos)
    assert torch.equal(a.view_as(ql), ql) and torch.equal(b.view_as(qr), qr)


# ---------------------------------------------------------------- append

APPENDS = [([1], [1]), ([3, 0, 70, 1], [3, 7, 200, 64]), ([8] * 40, [64 + 3 * i for i in range(40)]), ([700, 5], [700, 900])]


@pytest.mark.parametrize("given", [False, True], ids=["slots", "positions"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("counts,lens", APPENDS, ids=[f"{i}" for i in range(len(APPENDS))])
def test_append_parity(counts, lens, fp8, given):
    c = TU.case(counts, lens, "none", seed=41, pad=3)
    T, n = c["T"], int(c["offsets"][-1])
    g = torch.Generator().manual_seed(42)
    kv = (torch.randn(T, 576, generator=g) * torch.logspace(-3, 3, T)[:, None]).to(torch.bfloat16)
    gamma = (1 + 0.1 * torch.randn(512, generator=g)).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    if n > 4:
        pos[2] = -1
        kv[3, :512] = 0                                            # an all-zero latent
    width = 656 if fp8 else 576
    cache = torch.randint(0, 256, (c["pages"], 64, width), generator=g, dtype=torch.uint8) if fp8 else \
        torch.randn(c["pages"], 64, width, generator=g).to(torch.bfloat16)
    kvc, cc, d = kv.cuda(), cache.cuda(), TU.index_tensors(c)
    f = mla.cache_append_fp8 if fp8 else mla.cache_append
    st = f(kvc[:, :512], kvc[:, 512:], gamma.cuda(), cc, d["block_table"], d["seq_lens"], d["offsets"],
           positions=pos.cuda() if given else None)
    assert st.item() == 0
    slots = [s for s in OT.token_slots(c["block_table"], c["seq_lens"], c["offsets"]) if not (given and pos[s[0]] < 0)]
    at = np.array([r for _, r, _ in slots])
    toks = np.array([t for t, _, _ in slots])
    where = pos.numpy()[toks] if given else np.array([s for _, _, s in slots])
    lat, rope = OT.token_rows(f64(kv)[toks][:, :512], f64(kv)[toks][:, 512:], gamma.double().numpy(), where)
    got = cc.cpu().reshape(-1, width)
    same = np.ones(len(got), bool)
    same[at] = False
    assert torch.equal(got[same], cache.reshape(-1, width)[same])       # nothing else is written
    pair = np.repeat(np.abs(f64(kv)[toks][:, 512:]).reshape(-1, 32, 2).sum(-1), 2, axis=-1)
    if not fp8:
        r = f64(got[at])
        assert (np.abs(r[:, :512] - lat) <= (BF + 1e-5) * np.abs(lat)).all()
        assert (np.abs(r[:, 512:] - rope) <= BF * np.abs(rope) + 2e-5 * pair).all()
        return
    raw = got[at].numpy()
    s = raw[:, 640:644].copy().view("<f4").reshape(-1).astype(np.float64)
    top = np.abs(lat).max(1)
    assert (np.abs(s - np.where(top > 0, top / 448.0, 1.0)) <= 1e-5 * s).all()
    assert (raw[:, 644:] == 0).all()
    rows = OF.dequantize_cache(raw)
    assert (np.abs(rows[:, :512] - lat) <= (2.0 ** -4 + 1e-4) * np.abs(lat) + 2.0 ** -10 * s[:, None]).all()
    assert (np.abs(rows[:, 512:] - rope) <= (BF + 1e-4) * np.abs(rope) + 2e-5 * pair).all()


def test_append_bad_inputs_are_flagged_and_skipped():
    c = TU.case([2, 3, 2, 2], [1, 200, 64, 300], "none", seed=43)        # request 0: shorter than its tokens
    c["block_table"][2, 0] = -1
    c["block_table"][3, 4] = c["pages"]
    kv = torch.randn(9, 576, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(c["pages"], 64, 576, dtype=torch.bfloat16, device="cuda")
    d = TU.index_tensors(c)
    st = mla.cache_append(kv[:, :512], kv[:, 512:], gamma, cache, d["block_table"], d["seq_lens"], d["offsets"])
    assert st.item() == mla.MLA_DEV_BAD_SEQ_LEN | mla.MLA_DEV_BAD_PAGE
    written = (cache.view(-1, 576) != 0).any(-1).nonzero().view(-1).cpu().tolist()
    good = {int(c["block_table"][1][s // 64]) * 64 + s % 64 for s in (197, 198, 199)}
    good |= {int(c["block_table"][0][0]) * 64}                          # request 0's second token stands at slot 0
    assert set(written) == good
    off = torch.tensor([0, 5, 3, 7, 9], dtype=torch.int32, device="cuda")
    st = mla.cache_append(kv[:, :512], kv[:, 512:], gamma, cache, d["block_table"], d["seq_lens"], off)
    assert st.item() & mla.MLA_DEV_BAD_OFFSETS


# ---------------------------------------------------------------- commit

@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("layers", [None, 1, 5])
def test_commit_parity(fp8, layers):
    counts = [1, 6, 64, 64, 0, 9, 5, 33]
    lens = [1, 66, 64, 127, 30, 500, 5, 96]
    c = TU.case(counts, lens, "none", seed=51)
    rng = np.random.default_rng(52)
    paths, plens = np.full((8, 64), -5, np.int32), np.zeros(8, np.int32)
    for b, n in enumerate(counts):
        k = {2: 64, 3: 40, 6: 0}.get(b, min(n, int(rng.integers(1, 8))))
        plens[b] = k if n else 3                                  # of no request: not looked at
        paths[b, :k] = np.sort(rng.choice(max(n, 1), k, replace=False)) if n else 0
    width = 656 if fp8 else 576
    shape = ((layers,) if layers else ()) + (c["pages"], 64, width)
    g = torch.Generator().manual_seed(53)
    cache = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8) if fp8 else \
        torch.randn(shape, generator=g).to(torch.bfloat16)
    cc, d = cache.cuda(), TU.index_tensors(c)
    f = mla.cache_commit_fp8 if fp8 else mla.cache_commit
    new, st = f(cc, d["block_table"], d["seq_lens"], d["offsets"], torch.from_numpy(paths).cuda(), torch.from_numpy(plens).cuda())
    assert st.item() == 0
    bits = (lambda t: t) if fp8 else (lambda t: t.view(torch.int16))
    for got, was in zip(cc.cpu().reshape(-1, c["pages"] * 64, width), cache.reshape(-1, c["pages"] * 64, width)):
        want, lens_after = OT.commit(bits(was).numpy(), c["block_table"], c["seq_lens"], c["offsets"], paths, plens)
        assert np.array_equal(bits(got).numpy(), want)
    assert new.cpu().numpy().tolist() == lens_after.tolist()


def test_commit_bad_paths_leave_the_cache():
    counts, lens = [4] * 6, [100, 100, 2, 100, 100, 100]
    c = TU.case(counts, lens, "none", seed=54)
    c["block_table"][5, 1] = c["pages"] + 1
    paths = np.array([[0, 0], [0, 4], [0, 1], [1, 0], [-1, 2], [0, 1]], np.int32)
    plens = np.array([2, 2, 2, 2, 2, 2], np.int32)
    cache = torch.randn(c["pages"], 64, 576, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    cc, d = cache.cuda(), TU.index_tensors(c)
    new, st = mla.cache_commit(cc, d["block_table"], d["seq_lens"], d["offsets"], torch.from_numpy(paths).cuda(),
                               torch.from_numpy(plens).cuda())
    assert st.item() == mla.MLA_DEV_BAD_PATH | mla.MLA_DEV_BAD_SEQ_LEN | mla.MLA_DEV_BAD_PAGE
    assert torch.equal(cc.cpu(), cache) and new.cpu().tolist() == lens
    plens[:] = [5, 3, -1, 0, 1, 0]                                # longer than the tree, than max_path, negative
    paths[:] = 0
    new, st = mla.cache_commit(cc, d["block_table"], d["seq_lens"], d["offsets"], torch.from_numpy(paths).cuda(),
                               torch.from_numpy(plens).cuda())
    assert st.item() & mla.MLA_DEV_BAD_PATH
    assert torch.equal(cc.cpu(), cache) and new.cpu().tolist() == [100, 100, 2, 96, 97, 100]


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_a_speculative_step(fp8):
    """Query, append, attention, value projection, commit, then the next step's tokens: in one graph, against fp64."""
    counts, lens = [7, 12, 1], [90, 400, 64]
    c = TU.case(counts, lens, "tree", seed=61, spare=6)
    c["block_table"][2, 1] = c["order"][-1]                        # the next step's token needs a second page
    T = c["T"]
    _, _, cache = TU.tensors(c, seed=62, poison=False)
    g = torch.Generator().manual_seed(63)
    bf = torch.bfloat16
    q = torch.randn(T, 128, 192, generator=g).to(bf)
    kv = torch.randn(T, 576, generator=g).to(bf)
    w_uk = (torch.randn(128, 128, 512, generator=g) * 128 ** -0.5).to(bf)
    w_uv = (torch.randn(128, 128, 512, generator=g) * 512 ** -0.5).to(bf)
    gamma = torch.ones(512, dtype=bf)
    depth = [bin(int(m)).count("1") - 1 for m in c["masks"]]
    pos = np.concatenate([np.full(n, L - n) for n, L in zip(counts, lens)]) + np.array(depth)
    paths = np.zeros((3, 4), np.int32)
    plens = np.zeros(3, np.int32)
    for b, n in enumerate(counts):                                 # accept the deepest node's path
        t = max(range(int(c["offsets"][b]), int(c["offsets"][b + 1])), key=lambda i: (depth[i], i))
        way = [j for j in range(n) if int(c["masks"][t]) >> j & 1][:4]
        paths[b, :len(way)], plens[b] = way, len(way)
    cc = mla.quantize_cache_fp8(cache.cuda()) if fp8 else cache.cuda()
    start = cc.clone()
    d = TU.index_tensors(c)
    qc, kvc, wk, wv, gm = q.cuda(), kv.cuda(), w_uk.cuda(), w_uv.cuda(), gamma.cuda()
    posc, pc, plc = torch.from_numpy(pos.astype(np.int32)).cuda(), torch.from_numpy(paths).cuda(), torch.from_numpy(plens).cuda()
    table = mla.rope_table()
    append = mla.cache_append_fp8 if fp8 else mla.cache_append
    decode = mla.tree_decode_fp8 if fp8 else mla.tree_decode
    commit = mla.cache_commit_fp8 if fp8 else mla.cache_commit

    def step():
        ql, qr, st0 = mla.query(qc[..., :128], qc[..., 128:], wk, posc, table=table)
        st1 = append(kvc[:, :512], kvc[:, 512:], gm, cc, d["block_table"], d["seq_lens"], d["offsets"], positions=posc,
                     table=table)
        p = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=d["block_table"].shape[1])
        o, lse = decode(p, ql, qr, cc, d["block_table"], scale=SCALE)
        o_v, st2 = mla.epilog_uv(o.view(T, 1, 128, 512), wv)
        held = cc.clone()
        new, st3 = commit(cc, d["block_table"], d["seq_lens"], d["offsets"], pc, plc)
        return ql, qr, o, lse, o_v, held, new, p, (st0, st1, st2, st3)

    first = step()
    torch.cuda.synchronize()
    after = cc.clone()
    ql, qr, o, lse, o_v, held, new, p, sts = first
    assert mla.check(p) == 0 and all(s.item() == 0 for s in sts)
    rows = OF.dequantize_cache(held.cpu().numpy()) if fp8 else held.cpu()
    ref = OT.tree_decode(ql.cpu(), qr.cpu(), rows, c["block_table"], c["seq_lens"], c["offsets"], c["masks"], scale=SCALE)
    check_rows(o, lse, ref, slice(None))
    import oracle.epilog as OE  # noqa: F401  (the value projection has its own parity tests)
    bits = (lambda t: t) if fp8 else (lambda t: t.view(torch.int16))
    want, lens_after = OT.commit(bits(held.cpu()).reshape(-1, cc.shape[-1]).numpy(), c["block_table"], c["seq_lens"],
                                 c["offsets"], paths, plens)
    assert np.array_equal(bits(after.cpu()).reshape(-1, cc.shape[-1]).numpy(), want)
    assert new.cpu().tolist() == lens_after.tolist()
    # the same step, captured and replayed
    cc.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = step()
    for _ in range(2):
        cc.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cc, after)
        for a, b in zip(again[:7], first[:7]):
            assert torch.equal(a, b)
    # the next step: one token behind the accepted path sees it as a sequence
    n1 = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    sl = new + 1
    ql, qr, _ = mla.query(qc[:3, :, :128], qc[:3, :, 128:], wk, new, table=table)
    append(kvc[:3, :512], kvc[:3, 512:], gm, cc, d["block_table"], sl, n1, table=table)
    one = torch.ones(3, dtype=torch.int64, device="cuda")
    p = mla.tree_plan(sl, n1, one, max_pages_per_seq=d["block_table"].shape[1])
    o, lse = decode(p, ql, qr, cc, d["block_table"], scale=SCALE)
    assert mla.check(p) == 0
    rows = OF.dequantize_cache(cc.cpu().numpy()) if fp8 else cc.cpu()
    ref = OT.tree_decode(ql.cpu(), qr.cpu(), rows, c["block_table"], sl.cpu().numpy(), n1.cpu().numpy(),
                         np.ones(3, np.uint64), scale=SCALE)
    check_rows(o, lse, ref, slice(None))
