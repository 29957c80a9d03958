"""The tree step where it can go wrong silently: values that are not finite, memory that is short or shared
between streams, and every row of long calls (bounds as in test_gpu_tree.py)."""

import numpy as np
import pytest
import torch

import mla_decode_attention_02_gb300 as mla
import oracle.tree as OT
import tree_util as TU
from test_gpu_tree import BF, SCALE, check_rows, f64

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


# ---------------------------------------------------------------- latents that are not finite

def _append(fp8, kv, gamma, cache, d, **kw):
    f = mla.cache_append_fp8 if fp8 else mla.cache_append
    return f(kv[:, :512], kv[:, 512:], gamma, cache, d["block_table"], d["seq_lens"], d["offsets"], **kw)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("at", ["one", "all"])
def test_append_keeps_what_is_not_finite(fp8, value, at):
    """A token whose latent is not finite spoils its own row and the outputs of the nodes that see it, no other."""
    c = TU.case([6, 3], [70, 20], "self", seed=81)                 # every node sees its context and itself
    ql, qr, cache = TU.tensors(c, seed=82, quiet=True)
    g = torch.Generator().manual_seed(83)
    kv = torch.randn(c["T"], 576, generator=g).to(BF16)
    bad = [1, 4]
    for t in bad:
        kv[t, (slice(0, 512) if at == "all" else 37 * t)] = value
    gamma = (1 + 0.1 * torch.randn(512, generator=g)).to(BF16).cuda()
    d = TU.index_tensors(c)
    cc = mla.quantize_cache_fp8(cache.cuda()) if fp8 else cache.cuda()
    assert _append(fp8, kv.cuda(), gamma, cc, d).item() == 0
    slots = {t: r for t, r, _ in OT.token_slots(c["block_table"], c["seq_lens"], c["offsets"])}
    flat = cc.view(-1, cc.shape[-1])
    if fp8:
        codes = flat[:, :512].view(torch.float8_e4m3fn).float().cpu()
        scale = flat[:, 640:644].contiguous().view(torch.float32)[:, 0].cpu()
        for t in range(c["T"]):
            assert torch.isnan(codes[slots[t]]).all().item() is (t in bad), t
            assert torch.isnan(scale[slots[t]]).item() is (t in bad), t
    else:
        for t in range(c["T"]):
            assert torch.isnan(flat[slots[t], :512].float()).any().item() is (t in bad), t
    p = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=d["block_table"].shape[1])
    good = [t for t in range(c["T"]) if t not in bad]
    rows = _rows64(cc)
    ref = OT.tree_decode(ql, qr, rows, c["block_table"], c["seq_lens"], c["offsets"], c["masks"], scale=SCALE)
    for more in ({"scratch": False}, {"scratch": None}) if fp8 else ({},):
        f = mla.tree_decode_fp8 if fp8 else mla.tree_decode
        o, lse = f(p, ql.cuda(), qr.cuda(), cc, d["block_table"], scale=SCALE, **more)
        assert mla.check(p) == 0
        assert torch.isnan(o[bad].float()).any(-1).all() and torch.isnan(lse[bad]).all()
        check_rows(o[good], lse[good], tuple(x[good] for x in ref), slice(None))


def _rows64(cache):
    """fp64 rows of a cache of either kind, as a tensor of its shape."""
    if cache.dtype != torch.uint8:
        return cache.double().cpu()
    code, rope = cache[..., :512].view(torch.float8_e4m3fn), cache[..., 512:640].view(BF16)
    s = cache[..., 640:644].contiguous().view(torch.float32)
    return (torch.cat([code.float(), rope.float()], -1).double() * s.double()).cpu()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_append_of_zero_latents(fp8):
    """A zero latent is a zero row with any eps > 0; with eps = 0 it is 0 / 0 in either cache.  Zero weights: a zero row."""
    c = TU.case([3], [9], "none", seed=84)
    d = TU.index_tensors(c)
    kv = torch.randn(3, 576, generator=torch.Generator().manual_seed(85)).to(BF16)
    kv[1, :512] = 0
    ones, zeros = torch.ones(512, dtype=BF16, device="cuda"), torch.zeros(512, dtype=BF16, device="cuda")
    at = [r for _, r, _ in OT.token_slots(c["block_table"], c["seq_lens"], c["offsets"])]
    empty = torch.zeros(c["pages"], 64, 656 if fp8 else 576, dtype=torch.uint8 if fp8 else BF16, device="cuda")

    def rows(gamma, eps):
        cache = empty.clone()
        assert _append(fp8, kv.cuda(), gamma, cache, d, rms_eps=eps).item() == 0
        if fp8:
            assert (cache.view(-1, 656)[at][:, 644:] == 0).all()
        return _rows64(cache).view(-1, 576)[at]

    r = rows(ones, 1e-6)
    assert (r[1, :512] == 0).all() and torch.isfinite(r).all() and (r[0, :512] != 0).any()
    assert (r[:, 512:] != 0).all()                                # the rotary part stays
    r = rows(ones, 0.0)
    assert torch.isnan(r[1, :512]).all() and torch.isfinite(r[[0, 2]]).all()
    r = rows(zeros, 1e-6)
    assert (r[:, :512] == 0).all() and (r[:, 512:] != 0).all()


def test_fp8_append_of_a_weight_that_is_not_a_number():
    c = TU.case([2], [5], "none", seed=86)
    d = TU.index_tensors(c)
    kv = torch.randn(2, 576, generator=torch.Generator().manual_seed(87)).to(BF16).cuda()
    for rest in (1.0, 0.0):
        gamma = torch.full((512,), rest, dtype=BF16, device="cuda")
        gamma[300] = float("nan")
        cache = torch.zeros(c["pages"], 64, 656, dtype=torch.uint8, device="cuda")
        _append(True, kv, gamma, cache, d)
        at = [r for _, r, _ in OT.token_slots(c["block_table"], c["seq_lens"], c["offsets"])]
        assert torch.isnan(_rows64(cache).view(-1, 576)[at][:, 300]).all()


# ---------------------------------------------------------------- memory

def _wait_ms(ms):
    torch.cuda._sleep(int(ms * 2e6))


@pytest.mark.parametrize("kind", ["tree", "tree_fp8", "plain", "plain_fp8"])
@pytest.mark.parametrize("way", ["current", "given", "home"])
def test_a_dropped_plan_outlives_its_calls(kind, way):
    """A plan made on one stream and used on another ("current": the current one, "given": stream=) keeps its
    memory from reuse until that work is done; on one stream alone ("home") it is free for the next call at once."""
    c = TU.case([2, 2, 2], [90, 700, 64], "chain", seed=95)
    ql, qr, cache = TU.tensors(c, seed=96, quiet=True)
    d = TU.index_tensors(c)
    tree, fp8 = kind.startswith("tree"), kind.endswith("fp8")
    kv = mla.quantize_cache_fp8(cache.cuda()) if fp8 else cache.cuda()
    ql, qr = ql.cuda(), qr.cuda()
    table = torch.where(d["block_table"] == 1 << 30, -1, d["block_table"])
    if tree:
        plan = lambda **kw: mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=table.shape[1], **kw)  # noqa: E731
        f = mla.tree_decode_fp8 if fp8 else mla.tree_decode
        run = lambda p, **kw: f(p, ql, qr, kv, table, scale=SCALE, **kw)  # noqa: E731
    else:
        plan = lambda **kw: mla.plan(d["seq_lens"], s_q=2, max_pages_per_seq=table.shape[1], **kw)  # noqa: E731
        f = mla.decode_fp8 if fp8 else mla.decode
        run = lambda p, **kw: f(p, ql.view(3, 2, 128, 512), qr.view(3, 2, 128, 64), kv, table, scale=SCALE, **kw)  # noqa: E731
    want = [x.clone() for x in run(plan())]
    here, there = torch.cuda.current_stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    if way == "current":            # made where `there` is current, used here
        home, user, kw = there, here, {}
    elif way == "given":            # made here, used on a stream that the call names
        home, user, kw = here, there, {"stream": there}
    else:
        home, user, kw = here, here, {}
    user.wait_stream(home)
    with torch.cuda.stream(user):
        _wait_ms(400)
    with torch.cuda.stream(home):
        p = plan()
    user.wait_stream(home)
    run(p, out=out, lse=lse, **kw)
    at, n = p.workspace.data_ptr(), p.workspace.numel()
    del p
    assert not user.query()                                        # the call still waits
    with torch.cuda.stream(home):
        got = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(3)]
    again = [t.data_ptr() for t in got]
    assert not user.query()
    torch.cuda.synchronize()
    assert (at in again) is (way == "home")
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("kind", ["tree", "plain"])
def test_an_eager_plan_in_a_captured_decode(kind):
    """A plan made outside a graph serves the decode captured in it, over replays, and is dropped after."""
    c = TU.case([2, 2, 2], [90, 700, 64], "chain", seed=106)
    ql, qr, cache = TU.tensors(c, seed=107, quiet=True)
    d = TU.index_tensors(c)
    ql, qr, kv = ql.cuda(), qr.cuda(), cache.cuda()
    table = torch.where(d["block_table"] == 1 << 30, -1, d["block_table"])
    if kind == "tree":
        p = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=table.shape[1])
        run = lambda **kw: mla.tree_decode(p, ql, qr, kv, table, scale=SCALE, **kw)  # noqa: E731
    else:
        p = mla.plan(d["seq_lens"], s_q=2, max_pages_per_seq=table.shape[1])
        run = lambda **kw: mla.decode(p, ql.view(3, 2, 128, 512), qr.view(3, 2, 128, 64), kv, table, scale=SCALE, **kw)  # noqa: E731
    o, lse = run()
    want = [o.clone(), lse.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out=o, lse=lse)
    for _ in range(3):
        o.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and mla.check(p) == 0
    other = torch.cuda.CUDAGraph()                                  # dropped while another capture runs
    x = torch.zeros(8, device="cuda")
    del graph
    with torch.cuda.graph(other):
        x += 1
        del p, run
    other.replay()
    assert (x == 1).all()
    got = [torch.zeros(1 << 20, device="cuda") for _ in range(30)]
    torch.cuda.synchronize()
    assert not any(t.any() for t in got)


def test_a_decode_plan_made_on_a_given_stream():
    """plan(stream=s): the workspace comes from the current stream's memory and is written on s."""
    c = TU.case([2], [400], "chain", seed=97)
    d = TU.index_tensors(c)
    mla.plan(d["seq_lens"], s_q=2, max_pages_per_seq=d["block_table"].shape[1])
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _wait_ms(400)
    p = mla.plan(d["seq_lens"], s_q=2, max_pages_per_seq=d["block_table"].shape[1], stream=s)
    at, n = p.workspace.data_ptr(), p.workspace.numel()
    del p
    got = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(3)]
    assert not s.query() and at not in [t.data_ptr() for t in got]
    torch.cuda.synchronize()

@pytest.mark.parametrize("how", ["plain", "stream", "graph"])
def test_fp8_trees_run_where_memory_has_no_room_for_their_scratch(how):
    """A block table far wider than its requests asks for more scratch than there is: the same bits without it."""
    c = TU.case([5, 9, 16, 2], [70, 300, 129, 64], "tree", seed=91, width=8192)
    ql, qr, cache = TU.tensors(c, seed=92, quiet=True)
    d = TU.index_tensors(c)
    ql, qr, kv = ql.cuda(), qr.cuda(), mla.quantize_cache_fp8(cache.cuda())
    plan = lambda: mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=8192)  # noqa: E731
    p = plan()
    want = mla.tree_decode_fp8(p, ql, qr, kv, d["block_table"], scale=SCALE, scratch=False)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    need = p.batch * p.max_pages * mla.EXPANDED_PAGE_BYTES
    room = torch.cuda.memory_reserved() + (256 << 20)
    assert (1 << 30) < need <= mla.EXPAND_LIMIT_BYTES
    torch.cuda.set_per_process_memory_fraction(room / torch.cuda.get_device_properties(0).total_memory)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            torch.empty(need, dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream() if how == "stream" else None
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        call = lambda p: mla.tree_decode_fp8(p, ql, qr, kv, d["block_table"], scale=SCALE, stream=s)  # noqa: E731
        if how == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = [call(plan()) for _ in range(2)]
            graph.replay()
        else:
            got = [call(p) for _ in range(3)]
        torch.cuda.synchronize()
        for o, lse in got:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        if how != "graph":
            assert mla.check(p) == 0
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    o, lse = mla.tree_decode_fp8(plan(), ql, qr, kv, d["block_table"], scale=SCALE)       # and with it
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_fp8_trees_behind_a_wide_table_with_scratch():
    c = TU.case([3, 12], [200, 90], "tree", seed=93, width=300)
    ql, qr, cache = TU.tensors(c, seed=94, quiet=True)
    d = TU.index_tensors(c)
    kv = mla.quantize_cache_fp8(cache.cuda())
    p = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=300)
    room = torch.full((2 * 300 * mla.EXPANDED_PAGE_BYTES,), 0xFF, dtype=torch.uint8, device="cuda")
    ref = OT.tree_decode(ql, qr, _rows64(kv), c["block_table"], c["seq_lens"], c["offsets"], c["masks"], scale=SCALE)
    for scratch in (False, None, room):
        o, lse = mla.tree_decode_fp8(p, ql.cuda(), qr.cuda(), kv, d["block_table"], scale=SCALE, scratch=scratch)
        assert mla.check(p) == 0
        check_rows(o, lse, ref, slice(None))


# ---------------------------------------------------------------- marshalling

@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_calls_marshalled_in_python_are_the_same(fp8, monkeypatch):
    import mla_decode_attention_02_gb300._binding as binding
    c = TU.case([4, 7, 0, 9], [70, 200, 5, 64], "tree", seed=98, pad=1)
    _, _, cache = TU.tensors(c, seed=99, quiet=True)
    d = TU.index_tensors(c)
    g = torch.Generator().manual_seed(100)
    q = torch.randn(c["T"], 128, 192, generator=g).to(BF16).cuda()
    kv = torch.randn(c["T"], 576, generator=g).to(BF16).cuda()
    w = (torch.randn(128, 128, 512, generator=g) * 128 ** -0.5).to(BF16).cuda()
    pos = torch.arange(c["T"], dtype=torch.int32, device="cuda")
    paths = torch.tensor([[0, 3], [2, 5], [0, 0], [1, 8]], dtype=torch.int32, device="cuda")
    plens = torch.tensor([2, 2, 0, 2], dtype=torch.int32, device="cuda")
    start = mla.quantize_cache_fp8(cache.cuda()) if fp8 else cache.cuda()
    decode = mla.tree_decode_fp8 if fp8 else mla.tree_decode
    commit = mla.cache_commit_fp8 if fp8 else mla.cache_commit

    def step():
        cc = start.clone()
        ql, qr, s0 = mla.query(q[..., :128], q[..., 128:], w, pos)
        s1 = _append(fp8, kv, torch.ones(512, dtype=BF16, device="cuda"), cc, d, positions=pos)
        p = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=d["block_table"].shape[1])
        n = int(c["offsets"][-1])
        o, lse = (x[:n] for x in decode(p, ql, qr, cc, d["block_table"], scale=SCALE))
        held = cc.clone()
        new, s2 = commit(cc, d["block_table"], d["seq_lens"], d["offsets"], paths, plens)
        assert mla.check(p) == 0
        return ql, qr, o, lse, held, cc, new, s0, s1, s2

    assert type(binding._native()) is not type                    # the native module, not its stand-in
    native = step()
    monkeypatch.setattr(binding, "_host", binding._PythonOnly)
    for a, b in zip(native, step()):
        assert a.dtype == b.dtype and torch.equal(a.view(torch.uint8) if a.is_contiguous() else a, b.view(torch.uint8) if b.is_contiguous() else b)
    assert all(s.item() == 0 for s in native[-3:])


def test_bytes_of_any_shape_on_a_given_stream():
    """Workspace and scratch are bytes: their shape does not matter, with stream= as without."""
    c = TU.case([5, 9], [70, 300], "tree", seed=101)
    ql, qr, cache = TU.tensors(c, seed=102, quiet=True)
    d = TU.index_tensors(c)
    width = d["block_table"].shape[1]
    kv, qlc, qrc = mla.quantize_cache_fp8(cache.cuda()), ql.cuda(), qr.cuda()
    n = (mla.tree_workspace_size(2, c["T"], width) + 255) // 256
    room = 2 * width * mla.EXPANDED_PAGE_BYTES // 64
    s = torch.cuda.Stream()
    got = []
    for stream in (None, s):
        ws, scratch = (torch.empty(k, dtype=torch.uint8, device="cuda") for k in ((n, 16, 16), (room, 64)))
        s.wait_stream(torch.cuda.current_stream())
        p = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=width, workspace=ws, stream=stream)
        got.append(mla.tree_decode_fp8(p, qlc, qrc, kv, d["block_table"], scale=SCALE, scratch=scratch, stream=stream))
        torch.cuda.synchronize()
        assert mla.check(p) == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    with pytest.raises(TypeError, match="workspace"):
        mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=width, workspace=[1], stream=s)
    with pytest.raises(ValueError, match="table"):
        mla.query(torch.zeros(1, 128, 128, dtype=BF16, device="cuda"), torch.zeros(1, 128, 64, dtype=BF16, device="cuda"),
                  torch.zeros(128, 128, 512, dtype=BF16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                  table=torch.zeros(64), stream=s)


# ---------------------------------------------------------------- every row of long calls

@pytest.mark.parametrize("T", [81, 1537, 2049, 4097, 33000])
def test_every_row_of_many_queries(T):
    """The persistent kernel's rows, all tiles of all its CTAs, are those of calls of 80 tokens bit for bit."""
    g = torch.Generator(device="cuda").manual_seed(T)
    q = torch.randn(T, 128, 192, generator=g, device="cuda", dtype=BF16)
    w = torch.randn(128, 128, 512, generator=g, device="cuda", dtype=BF16) * 128 ** -0.5
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[::7] = -1                                                  # left out, in every tile
    ql = torch.full((T, 128, 512), 7.0, dtype=BF16, device="cuda")
    qr = torch.full((T, 128, 64), 7.0, dtype=BF16, device="cuda")
    for _ in range(2):                                             # the second over the first one's rows
        _, _, st = mla.query(q[..., :128], q[..., 128:], w, pos, q_latent=ql, q_rope=qr)
        assert st.item() == 0
    assert (ql[::7] == 7).all() and (qr[::7] == 7).all()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for at in range(0, T, 80):
        few = slice(at, min(at + 80, T))
        a, b, _ = mla.query(q[few, :, :128], q[few, :, 128:], w, pos[few])
        keep = pos[few] >= 0
        wrong += (ql[few] != a).flatten(1).any(1).logical_and(keep).sum()
        wrong += (qr[few] != b).flatten(1).any(1).logical_and(keep).sum()
    assert wrong.item() == 0


# ---------------------------------------------------------------- the step's value projection

@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_the_value_projection_of_a_tree(fp8):
    """Heads of a drafted tree's attention, projected: against fp64 from the outputs, and from the cache itself."""
    import oracle.epilog as OE
    c = TU.case([7, 12, 1], [90, 400, 64], "tree", seed=103)
    ql, qr, cache = TU.tensors(c, seed=104, quiet=True)
    d = TU.index_tensors(c)
    kv = mla.quantize_cache_fp8(cache.cuda()) if fp8 else cache.cuda()
    w = (torch.randn(128, 128, 512, generator=torch.Generator().manual_seed(105)) * 512 ** -0.5).to(BF16)
    p = mla.tree_plan(d["seq_lens"], d["offsets"], d["masks"], max_pages_per_seq=d["block_table"].shape[1])
    f = mla.tree_decode_fp8 if fp8 else mla.tree_decode
    o, _ = f(p, ql.cuda(), qr.cuda(), kv, d["block_table"], scale=SCALE)
    o_v, st = mla.epilog_uv(o.view(c["T"], 1, 128, 512), w.cuda())
    assert st.item() == 0 and mla.check(p) == 0
    got = f64(o_v).reshape(c["T"], 128, 128)
    # one bf16 rounding and 512 fp32 products and sums
    ref, size = OE.uv_project(o, w), OE.uv_project(np.abs(f64(o)), np.abs(f64(w)))
    near = BF * np.abs(ref) + 512 * 2.0 ** -24 * size + 1e-6
    assert (np.abs(got - ref) <= near).all()
    # and the attention's own bound (test_gpu_tree.py) carried through the projection
    want, _, spread = OT.tree_decode(ql, qr, _rows64(kv), c["block_table"], c["seq_lens"], c["offsets"], c["masks"], scale=SCALE)
    far = OE.uv_project((2 * BF + 2.4e-3) * spread + BF * np.abs(want) + 1e-6, np.abs(f64(w)))
    assert (np.abs(got - OE.uv_project(want, w)) <= near + far).all()
