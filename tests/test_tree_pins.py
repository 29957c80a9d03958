"""CPU tests of the tree step: the oracle against the mathematics, the planner's schedule, the refusals."""

import ctypes

import numpy as np
import pytest
import torch

import mla_decode_attention_02_gb300 as mla
import mla_decode_attention_02_gb300._binding as binding
import oracle
import oracle.prolog as OP
import oracle.tree as OT
import tree_util as TU

SCALE = mla.DEFAULT_SCALE


# ---------------------------------------------------------------- the oracle

def test_oracle_tree_chain_equals_causal_decode():
    """A chain of two nodes is the s_q = 2 decode."""
    c = TU.case([2, 2], [70, 3], "chain", seed=1)
    ql, qr, cache = TU.tensors(c, seed=1, quiet=True)
    o, lse, _ = OT.tree_decode(ql, qr, cache, c["block_table"], c["seq_lens"], c["offsets"], c["masks"], scale=SCALE)
    ref, ref_lse = oracle.decode(ql.view(2, 2, 128, 512), qr.view(2, 2, 128, 64), cache, c["block_table"],
                                 c["seq_lens"], s_q=2, scale=SCALE)
    assert np.abs(o.reshape(ref.shape) - ref).max() < 1e-12
    assert np.abs(lse.reshape(ref_lse.shape) - ref_lse).max() < 1e-12


def test_oracle_tree_path_equals_its_own_sequence():
    """A node sees what the sequence context + its path would see."""
    c = TU.case([6], [80], "tree", seed=3)
    ql, qr, cache = TU.tensors(c, seed=3)
    o, lse, _ = OT.tree_decode(ql, qr, cache, c["block_table"], c["seq_lens"], c["offsets"], c["masks"], scale=SCALE)
    rows = OT.keys(cache, c["block_table"][0], 80)
    for t in range(6):
        path = [j for j in range(6) if int(c["masks"][t]) >> j & 1]
        assert path[-1] == t
        r = np.concatenate([rows[:74], rows[[74 + j for j in path]]])
        x = SCALE * (np.concatenate([OP._f64(ql[t]), OP._f64(qr[t])], 1) @ r.T)
        w = np.exp(x - x.max(1, keepdims=True))
        assert np.abs(w @ r[:, :512] / w.sum(1, keepdims=True) - o[t]).max() < 1e-12
        assert np.abs(np.log(np.exp(x).sum(1)) - lse[t]).max() < 1e-11


def test_oracle_empty_row():
    c = TU.case([3], [3], "none", seed=4)
    ql, qr, cache = TU.tensors(c, seed=4)
    o, lse, _ = OT.tree_decode(ql, qr, cache, c["block_table"], c["seq_lens"], c["offsets"], c["masks"], scale=SCALE)
    assert (o == 0).all() and (lse == -np.inf).all()


def test_oracle_token_rows_equal_the_prolog():
    """Appended rows at their slots are the prolog's cache rows."""
    g = torch.Generator().manual_seed(5)
    B, S = 2, 2
    lat, pe = torch.randn(B, S, 512, generator=g), torch.randn(B, S, 64, generator=g)
    gamma = torch.randn(512, generator=g)
    table, lens = np.array([[1, 0], [2, 3]], np.int32), np.array([65, 2], np.int32)
    _, _, cache = OP.prolog(torch.zeros(B, S, 128, 128), torch.zeros(B, S, 128, 64), lat, pe, torch.zeros(128, 128, 512),
                            gamma, np.zeros((4, 64, 576)), table, lens)
    off = np.array([0, 2, 4])
    slots = OT.token_slots(table, lens, off)
    c, k = OT.token_rows(lat.view(-1, 512), pe.view(-1, 64), gamma, [s for _, _, s in slots])
    for t, row, _ in slots:
        assert np.array_equal(cache.reshape(-1, 576)[row], np.concatenate([c[t], k[t]]))


def test_oracle_commit_moves_the_path():
    rows = np.arange(3 * 64 * 2).reshape(3 * 64, 2)
    table, lens, off = np.array([[2, 0]]), [66], [0, 6]       # tree slots 60 .. 65 over two pages
    new, n = OT.commit(rows, table, lens, off, [[0, 2, 5]], [3])
    assert n[0] == 63
    assert (new[2 * 64 + 60] == rows[2 * 64 + 60]).all()
    assert (new[2 * 64 + 61] == rows[2 * 64 + 62]).all()
    assert (new[2 * 64 + 62] == rows[0 * 64 + 1]).all()
    changed = np.flatnonzero((new != rows).any(1))
    assert changed.tolist() == [2 * 64 + 61, 2 * 64 + 62]


# ---------------------------------------------------------------- the planner

def _check_plan(c, units, max_pages=None):
    mp = c["block_table"].shape[1] if max_pages is None else max_pages
    p = mla.tree_plan_host(c["seq_lens"], c["offsets"], c["masks"], max_pages_per_seq=mp, num_units=units)
    items, T = p["items"], c["T"]
    assert p["header"]["num_parts"] <= 2 * units
    assert (np.diff(p["item_unit"]) >= 0).all()
    ub = p["unit_begin"]
    assert ub[0] == 0 and ub[-1] == len(items)
    for u in range(units):
        assert (p["item_unit"][ub[u]:ub[u + 1]] == u).all()
    parts = []
    for t in range(T):
        mine = items[items[:, 0] == t]
        b = int(np.searchsorted(c["offsets"], t, side="right")) - 1
        if t >= c["offsets"][-1]:
            assert len(mine) == 0 and p["row_nparts"][t] == -2
            continue
        n, L = int(c["offsets"][b + 1] - c["offsets"][b]), int(c["seq_lens"][b])
        if L < n or L > mp * 64:
            assert len(mine) == 0 and p["row_nparts"][t] == 0
            continue
        seen = np.flatnonzero(OT.visible(L, n, c["masks"][t]))
        row = p["tree_rows"][t]
        assert row["req"] == b and row["context"] == L - n
        assert int(row["mask"]) == int(c["masks"][t]) & ((1 << n) - 1)
        if len(seen) == 0:
            assert len(mine) == 0 and p["row_nparts"][t] == -1
            continue
        assert p["row_nparts"][t] == len(mine)
        assert (p["tree_items"][items[:, 0] == t] == row).all()
        assert p["tree_pages"][b] >= (seen[-1] + 64) // 64
        at = 0
        for i, (_, k0, k1, part) in enumerate(mine):
            assert k0 == at and k1 > k0 and (k0 % 64 == 0)
            # an item's first page holds a visible key
            assert ((seen >= k0) & (seen < min(k0 + 64, k1))).any()
            # masked slots lie in the item's last two pages
            pages = (k1 - k0 + 63) // 64
            hidden = np.setdiff1d(np.arange(k0, k1), seen)
            assert (hidden >= k0 + 64 * (pages - 2)).all()
            if i < len(mine) - 1:
                assert k1 % 64 == 0
            assert (part >= 0) == (len(mine) > 1)
            parts += [part] if part >= 0 else []
            at = k1
        assert at == seen[-1] + 1
    assert sorted(parts) == list(range(p["header"]["num_parts"]))
    return p


@pytest.mark.parametrize("units", [1, 3, 76])
def test_plan_covers_the_visible_keys(units):
    rng = np.random.default_rng(units)
    for trial in range(30):
        B = int(rng.integers(1, 7))
        counts = [int(rng.integers(0, 65)) if rng.random() < 0.8 else 0 for _ in range(B)]
        lens = [n + int(rng.choice([0, 1, 63, 64, 65, int(rng.integers(0, 6000))])) for n in counts]
        kinds = [str(rng.choice(["chain", "tree", "self", "bits", "none", "all"])) for _ in range(B)]
        c = TU.case(counts, lens, kinds, seed=trial, pad=int(rng.integers(0, 4)) + (sum(counts) == 0))
        _check_plan(c, units)


def test_plan_flags_bad_lengths_and_offsets():
    c = TU.case([4, 4, 4], [100, 3, 2000], "tree", seed=7)
    p = _check_plan(c, 76, max_pages=4)
    assert p["header"]["status"] == mla.MLA_DEV_BAD_SEQ_LEN
    for off in ([1, 4, 8, 12], [0, 8, 4, 12], [0, 4, 8, 13], [0, 4, 8, -1]):
        p = mla.tree_plan_host(c["seq_lens"], off, c["masks"], max_pages_per_seq=40, num_units=76)
        assert p["header"]["status"] == mla.MLA_DEV_BAD_OFFSETS
        assert (p["row_nparts"] == 0).all() and len(p["items"]) == 0
    c = TU.case([65], [100], "chain", seed=8)       # more than 64 nodes
    p = mla.tree_plan_host(c["seq_lens"], c["offsets"], c["masks"], max_pages_per_seq=2, num_units=76)
    assert p["header"]["status"] == mla.MLA_DEV_BAD_OFFSETS


# ---------------------------------------------------------------- refusals

def _ragged(batch=2, tokens=8, heads=128, page=64, max_pages=4, flags=0):
    return binding._Ragged(batch, tokens, heads, page, max_pages, flags)


BAD_RAGGED = [(None, 1), (_ragged(batch=0), 1), (_ragged(tokens=0), 1), (_ragged(max_pages=0), 1), (_ragged(flags=2), 1),
              (_ragged(heads=64), 2), (_ragged(page=32), 2), (_ragged(tokens=1 << 24), 2), (_ragged(batch=1 << 25, max_pages=1), 2),
              (_ragged(batch=1, max_pages=1 << 25), 2), (_ragged(batch=1 << 10, max_pages=1 << 21), 2)]


def _ref(prob):
    return ctypes.byref(prob) if prob is not None else None


def test_entry_points_refuse_before_any_cuda_call():
    lib = mla.load_library()
    A = 0x10000            # an aligned address that is never dereferenced

    def append(prob=_ragged(), lat=A, ls=576, pe=A, ks=576, gamma=A, eps=1e-6, table=A, pos=A, cache=A, pages=8,
               bt=A, sl=A, off=A, st=A, name="mla_cache_append"):
        return getattr(lib, name)(_ref(prob), lat, ls, pe, ks, gamma, eps, table, pos, cache, pages, bt, sl, off, st, None)

    def query(T=4, qn=A, s=(24576, 192, 24576, 192), pe=A, w=A, table=A, pos=A, ql=A, qr=A, st=A):
        return lib.mla_query(T, qn, s[0], s[1], pe, s[2], s[3], w, table, pos, ql, qr, st, None)

    def plan(prob=_ragged(), sl=A, off=A, m=A, ws=A, n=1 << 30):
        return lib.mla_tree_plan(_ref(prob), sl, off, m, ws, n, None)

    def decode(prob=_ragged(), ql=A, qr=A, kv=A, pages=8, bt=A, scale=0.07, o=A, lse=A, ws=A, n=1 << 30,
               scratch=None, room=0, name="mla_tree_decode"):
        more = (scratch, room) if name == "mla_tree_decode_fp8" else ()
        return getattr(lib, name)(_ref(prob), ql, qr, kv, pages, bt, scale, o, lse, ws, n, *more, None)

    def commit(prob=_ragged(), kv=A, layers=2, stride=8 * 64 * 1152, row=1152, pages=8, bt=A, sl=A, off=A, paths=A,
               mp=4, pl=A, new=A + 64, st=A):
        return lib.mla_cache_commit(_ref(prob), kv, layers, stride, row, pages, bt, sl, off, paths, mp, pl, new, st, None)

    for prob, want in BAD_RAGGED:
        for f in (append, plan, decode, commit):
            assert f(prob=prob) == want, (f.__name__, want)
    assert append(prob=_ragged(flags=1)) == 1 and commit(prob=_ragged(flags=1)) == 1      # a decode flag
    assert plan(prob=_ragged(flags=1), n=64) == 3 and decode(prob=_ragged(flags=1), n=64) == 3
    for name in ("mla_cache_append", "mla_cache_append_fp8"):
        for key in ("lat", "pe", "gamma", "table", "cache", "bt", "sl", "off", "st"):
            assert append(**{key: None, "name": name}) == 1, key
            assert append(**{key: A + 2, "name": name}) == 1, key
        assert append(pos=A + 2, name=name) == 1
        for key in ("ls", "ks"):
            for bad in (0, -8, 4, 577, 1 << 31):
                assert append(**{key: bad, "name": name}) == 1, bad
        for bad in (-1.0, float("nan"), float("inf")):
            assert append(eps=bad, name=name) == 1
        assert append(pages=0, name=name) == 1 and append(pages=1 << 31, name=name) == 1
    assert query(T=0) == 1 and query(T=1 << 24) == 2
    for key in ("qn", "pe", "w", "table", "pos", "ql", "qr", "st"):
        assert query(**{key: None}) == 1, key
        assert query(**{key: A + 2}) == 1, key
    for i in range(4):
        for bad in (0, -8, 12, 1 << 31):
            s = [24576, 192, 24576, 192]
            s[i] = bad
            assert query(s=s) == 1, s
    for key in ("sl", "off", "m", "ws"):
        assert plan(**{key: None}) == 1 and plan(**{key: A + 2}) == 1, key
    assert plan(n=64) == 3
    for name in ("mla_tree_decode", "mla_tree_decode_fp8"):
        for key in ("ql", "qr", "kv", "bt", "o", "lse", "ws"):
            assert decode(**{key: None, "name": name}) == 1 and decode(**{key: A + 2, "name": name}) == 1, key
        for bad in (0.0, -1.0, float("nan"), float("inf")):
            assert decode(scale=bad, name=name) == 1
        assert decode(pages=0, name=name) == 1 and decode(n=1024, name=name) == 3
    for key in ("kv", "bt", "sl", "off", "paths", "pl", "new", "st"):
        assert commit(**{key: None}) == 1 and commit(**{key: A + 2}) == 1, key
    assert commit(new=A) == 1                                   # new_seq_lens is seq_lens
    assert commit(layers=0) == 1 and commit(row=1024) == 1 and commit(pages=0) == 1
    assert commit(mp=0) == 1 and commit(mp=65) == 1
    assert commit(stride=8 * 64 * 1152 + 8) == 1 and commit(stride=8 * 64 * 1152 - 16) == 1
    assert decode(scratch=A + 8, room=1 << 30, name="mla_tree_decode_fp8") == 1
    assert decode(scratch=A, room=2 * 4 * mla.EXPANDED_PAGE_BYTES - 1, name="mla_tree_decode_fp8") == 3
    assert decode(prob=_ragged(batch=65536), scratch=A, room=1 << 40, name="mla_tree_decode_fp8") == 2
    n = ctypes.c_size_t(0)
    assert lib.mla_tree_scratch_size(_ref(_ragged()), ctypes.byref(n)) == 0 and n.value == 8 * mla.EXPANDED_PAGE_BYTES
    assert lib.mla_tree_scratch_size(_ref(_ragged()), None) == 1 and lib.mla_tree_scratch_size(None, ctypes.byref(n)) == 1
    assert lib.mla_tree_workspace_size(None, ctypes.byref(n)) == 1
    assert lib.mla_tree_workspace_size(_ref(_ragged()), None) == 1


def test_binding_refuses_wrong_tensors():
    cpu = torch.zeros(4, 128, 192, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mla.query(cpu[..., :128], cpu[..., 128:], None, None)
    with pytest.raises(TypeError, match="bfloat16"):
        mla.query(cpu.float()[..., :128], cpu[..., 128:], None, None)
    with pytest.raises(ValueError, match="q_nope"):
        mla.query(cpu[:0, :, :128], cpu[:0, :, 128:], None, None)
    with pytest.raises(ValueError, match="kv_latent"):
        mla.cache_append(cpu, cpu, None, None, None, None, None)
    with pytest.raises(TypeError, match="kv_latent"):
        mla.cache_append(None, cpu, None, None, None, None, None)
    with pytest.raises(TypeError, match="int32"):
        mla.tree_plan(torch.zeros(2), None, None, max_pages_per_seq=1)
    with pytest.raises(ValueError, match="CUDA"):
        mla.cache_commit(None, torch.zeros(1, 1, dtype=torch.int32), None, None, None, None)


def test_native_marshalling_leaves_what_is_not_plain():
    """The C++ marshalling takes CUDA tensors only; anything else is the Python checks' to name."""
    h = binding._native()
    t = torch.zeros(1, dtype=torch.int32)
    assert h.query(*[t] * 8) is None and h.query() is None
    assert h.append(False, *[t] * 11) is None
    assert h.append(False, *[None] * 11) is None
    assert h.tree_plan(t, t, t, 1, None) is None
    assert h.tree_decode(1, 1, 1, t, t, t, t, t, 1.0, None, None, 0, False, None) is None
    assert h.commit(False, *[t] * 8) is None and h.commit(*[object()] * 9) is None
    with pytest.raises(TypeError):
        h.bind(1)
    with pytest.raises(ValueError):
        h.bind(*[0] * len(binding._HOST_ENTRIES))


def test_scratch_is_a_tensor_or_nothing():
    """A number of bytes is no scratch (0 ran without one, others were allocated)."""
    p = mla.TreePlan(1, 2, 4, torch.zeros(64, dtype=torch.uint8))
    for bad in (0, 1, 1 << 20, True, "room", [1]):
        with pytest.raises(TypeError, match="scratch"):
            mla.tree_decode_fp8(p, None, None, None, None, scratch=bad)
    with pytest.raises(TypeError, match="q_latent"):
        mla.tree_decode_fp8(p, None, None, None, None, scratch=False)


def test_arguments_of_no_device_on_a_given_stream():
    """What is no CUDA tensor is not recorded on the stream: the argument's own check names it."""
    class Stream:
        device = torch.device("cuda", 0)
        cuda_stream = 0
    cpu = torch.zeros(4)
    assert binding._launch_on(0, Stream(), cpu, None, False, "text", 7) is not None
    with pytest.raises(ValueError, match="cuda:1"):
        binding._launch_on(1, Stream(), cpu)
