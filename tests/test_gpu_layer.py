"""GPU parity of rotary positions, residual norms and a whole chunk step with the 64-bit oracle.

Tolerances (a bf16 rounding is off by at most BF = 2^-8 of the value):

* rotate: one rounding; the sine and cosine are good to 1e-6 and the angle to 1e-6 rad below position 2^20, 1e-5 below
  2^31 (mla_prolog.cu), times the pair's size and the magnitude: |y - ref| <= BF |ref| + e m (|x_a| + |x_b|), with
  e = 3e-6 below 2^20 and 2e-5 beyond.
* norm: z in fp32 (half a step of its own: 2^-24), a sum of N squares (at most N 2^-24 of itself, in practice far less),
  rsqrt and products a few 2^-24: below 1e-5 relative for the sizes here (a sum of 32 partial sums per thread and
  warps), then one rounding: BF for bf16; a code is off by half an e4m3 step, 2^-4 of the value or 2^-10 of the scale, a
  tie by the 1e-5 more.
"""

import math

import pytest
import torch

import mla_decode_attention_02_gb300 as mla
import oracle.chunk as OC

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


def normal(*shape, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def check_rotated(y, x, positions, rate, half, magnitude=1.0, inverse=False, far=False):
    ref = OC.rotate(x, positions, rate, half=half, magnitude=magnitude, inverse=inverse)
    a = x.double().abs()
    n = a.shape[-1] // 2
    size = (a[..., :n] + a[..., n:]).repeat(1, 1, 2) if half else (a[..., 0::2] + a[..., 1::2]).repeat_interleave(2, -1)
    over = (y.double() - ref).abs() - (BF * ref.abs() + (2e-5 if far else 3e-6) * magnitude * size + 1e-30)
    assert over.max() <= 0, over.max()


@pytest.mark.parametrize("half", [False, True], ids=["interleaved", "half"])
@pytest.mark.parametrize("tokens,heads,dims", [(1, 1, 16), (1, 128, 64), (3, 7, 32), (5, 128, 128), (2, 3, 256), (65, 33, 64),
                                               (300, 128, 64), (4, 129, 16), (1, 700, 64)])
def test_rotate(tokens, heads, dims, half):
    g = torch.Generator().manual_seed(1)
    table = mla.rope_table_scaled(dims=dims)
    rate = OC.rates(dims)
    x = normal(tokens, heads, dims, seed=2)
    positions = torch.randint(0, 1 << 20, (tokens,), generator=g, dtype=torch.int32).cuda()
    layout = "half" if half else "interleaved"
    y = mla.rotate(x, positions, table=table, layout=layout)
    check_rotated(y, x, positions, rate, half)
    back = mla.rotate(x, positions, table=table, layout=layout, inverse=True, magnitude=1.25)
    check_rotated(back, x, positions, rate, half, magnitude=1.25, inverse=True)


@pytest.mark.parametrize("half", [False, True], ids=["interleaved", "half"])
def test_rotate_part_of_each_head_in_place(half):
    q = normal(9, 128, 192, seed=3)
    kept = q.clone()
    positions = torch.tensor([0, 1, 5, -1, 163839, 1 << 20, (1 << 31) - 1, -7, 77], dtype=torch.int32, device="cuda")
    table = mla.rope_table_scaled(factor=40.0)
    view = q[..., 128:]
    assert mla.rotate(view, positions, table=table, layout="half" if half else "interleaved", out=view) is view
    assert torch.equal(q[..., :128], kept[..., :128])
    left_out = positions < 0
    assert torch.equal(q[left_out], kept[left_out])
    keep = ~left_out
    check_rotated(q[keep][..., 128:], kept[keep][..., 128:], positions[keep], OC.rates(64, factor=40.0), half, far=True)
    assert torch.equal(q[0, :, 128:], kept[0, :, 128:])                    # position 0 turns nothing


def test_rotate_into_a_strided_output():
    x = normal(6, 5, 64, seed=4)
    positions = torch.arange(6, dtype=torch.int32, device="cuda") * 1000
    wide = torch.full((6, 9, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    mla.rotate(x, positions, table=mla.rope_table(), out=wide[:, 2:7, 16:80])
    check_rotated(wide[:, 2:7, 16:80], x, positions, OC.rates(64), False)
    wide[:, 2:7, 16:80] = 7
    assert (wide == 7).all()


def test_a_rotation_and_its_inverse_are_each_others_gradient():
    """<R x, g> = <x, R^T g>: the inverse is the gradient, also against differences of the rotation itself."""
    table, rate = mla.rope_table_scaled(factor=4.0), OC.rates(64, factor=4.0)
    x, g = normal(4, 8, 64, seed=5), normal(4, 8, 64, seed=6)
    positions = torch.tensor([3, 50, 7000, 100000], dtype=torch.int32, device="cuda")
    for layout, half in (("interleaved", False), ("half", True)):
        grad = mla.rotate(g, positions, table=table, layout=layout, inverse=True, magnitude=1.1)
        check_rotated(grad, g, positions, rate, half, magnitude=1.1, inverse=True)
        xd = x.double().requires_grad_()
        (OC.rotate(xd, positions, rate, half=half, magnitude=1.1) * g.double()).sum().backward()
        assert (grad.double() - xd.grad).abs().max() <= BF * xd.grad.abs().max() + 1e-4
        step = 0.5 * g                                     # (exact in bf16; the rotation is linear)
        up = mla.rotate(x + step, positions, table=table, layout=layout, magnitude=1.1).double()
        down = mla.rotate(x - step, positions, table=table, layout=layout, magnitude=1.1).double()
        diff = ((up - down) * g.double()).sum()
        want = ((x + step).double() - (x - step).double()) * grad.double()
        # each of 2048 products is off by three roundings of values below 8 (BF 8 sqrt(2) each), times |g| below 5
        assert abs(diff - want.sum()) <= 2048 ** 0.5 * 3 * BF * 8 * 1.5 * 5


@pytest.mark.parametrize("base,dims,factor,original,fast,slow", [
    (10000.0, 64, 1.0, 4096, 32.0, 1.0), (10000.0, 64, 40.0, 4096, 32.0, 1.0), (10000.0, 128, 4.0, 8192, 32.0, 1.0),
    (500000.0, 16, 8.0, 131072, 32.0, 1.0), (10000.0, 256, 16.0, 64, 32.0, 1.0), (10000.0, 32, 2.0, 4096, 4.0, 4.0),
    (10000.0, 64, 1e6, 1, 32.0, 1.0)])
def test_scaled_table(base, dims, factor, original, fast, slow):
    t = mla.rope_table_scaled(base, dims=dims, factor=factor, original_positions=original, beta_fast=fast, beta_slow=slow)
    turns = t[:dims // 2].double() + t[dims // 2:].double()
    ref = OC.rates(dims, base, factor, original, fast, slow).cuda() / (2 * math.pi)
    # fp64 pow and a handful of fp64 steps, then two floats: 2^-48
    assert ((turns - ref).abs() <= 1e-13 * ref).all()
    if factor == 1.0 and dims == 64:
        plain = mla.rope_table(base)
        assert ((turns - plain[:32].double() - plain[32:].double()).abs() <= 1e-13 * turns).all()


def test_scaled_table_in_the_other_entry_points():
    """Queries and appended rows turn by the scaled table as rotate does."""
    table = mla.rope_table_scaled(factor=40.0)
    q, w_uk = normal(3, 128, 192, seed=7), normal(128, 128, 512, seed=8, std=128 ** -0.5)
    positions = torch.tensor([5, 4097, 100001], dtype=torch.int32, device="cuda")
    _, q_rope, _ = mla.query(q[..., :128], q[..., 128:], w_uk, positions, table=table)
    assert torch.equal(q_rope, mla.rotate(q[..., 128:], positions, table=table))


def check_norm(x, residual, weight, out, kept, eps):
    y, z = OC.residual_norm(x, residual, weight, eps)
    assert ((out.double() - y).abs() <= (BF + 1e-5) * y.abs() + 1e-30).all()
    if residual is not None:
        assert ((kept.double() - z).abs() <= (BF + 1e-6) * z.abs()).all()


@pytest.mark.parametrize("tokens,hidden", [(1, 8), (3, 64), (2, 512), (5, 1000), (1, 7168), (67, 7168), (700, 1536), (2, 2056), (3, 16384),
                                           (2, 10240), (4, 5128), (2, 12296), (3, 14344)])
def test_residual_norm(tokens, hidden):
    x, r, w = normal(tokens, hidden, seed=9), normal(tokens, hidden, seed=10, std=3.0), normal(hidden, seed=11)
    out, kept = mla.residual_norm(x, r, w, rms_eps=1e-6)
    check_norm(x, r, w, out, kept, 1e-6)
    alone, none = mla.residual_norm(x, None, w, rms_eps=0.5)
    assert none is None
    check_norm(x, None, w, alone, None, 0.5)
    y, z = OC.residual_norm(x, r, w, 1e-6)
    for group in (0, 128):
        codes, scales, kept8 = mla.residual_norm_fp8(x, r, w, group=group, rms_eps=1e-6)
        assert torch.equal(kept8, kept)
        ref, full = OC.group_scales(y, group)
        assert scales.shape == ref.shape and ((scales.double() - ref).abs() <= 1e-5 * ref).all()
        off = (codes.double() - y / full).abs()
        assert (off <= (2.0 ** -4 + 2e-5) * (y / full).abs().clamp(min=2.0 ** -6) + 1e-9).all()
        assert ((codes.double().abs() <= 448).all())


def test_norm_strides_in_place_and_streams():
    wide = normal(33, 8000, seed=12)
    x, r, w = wide[:, 8:7176], normal(33, 7168, seed=13), normal(7168, seed=14)
    out, kept = mla.residual_norm(x.contiguous(), r, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, k2 = mla.residual_norm(x, r, w, stream=s)
    s.synchronize()
    assert torch.equal(out, o2) and torch.equal(kept, k2)
    mine = r.clone()
    o3, k3 = mla.residual_norm(x, mine, w, residual_out=mine)
    assert k3 is mine and torch.equal(o3, out) and torch.equal(mine, kept)
    c, sc, _ = mla.residual_norm_fp8(x, r, w)
    c2, sc2, k4 = mla.residual_norm_fp8(x, r, w, stream=s)
    s.synchronize()
    assert torch.equal(c.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(sc, sc2) and torch.equal(k4, kept)


def test_norm_of_zeros_tiny_large_and_broken_rows():
    N = 512
    x = torch.zeros(8, N, dtype=torch.bfloat16, device="cuda")
    x[1, 5] = float("nan")
    x[2, 300] = float("inf")
    x[3] = 1e-38                                           # squares vanish: eps alone is left
    x[4] = 3e38                                            # their sum passes fp32's range: the norm is 0
    x[5, :128] = 2.0
    x[6] = -0.0
    x[7, 1] = 1e-40
    w = torch.ones(N, dtype=torch.bfloat16, device="cuda")
    r = torch.zeros_like(x)
    out, kept = mla.residual_norm(x, r, w, rms_eps=1e-6)
    assert torch.equal(kept[3:6], x[3:6]) and (out[0] == 0).all() and (out[6] == 0).all() and (out[4] == 0).all()
    assert torch.isnan(out[1].float()).all() and torch.isnan(out[2, 300].float())
    alone, _ = mla.residual_norm(x[6:7], None, w)
    assert torch.equal(alone.view(torch.int16), x[6:7].view(torch.int16))            # (negative zeros stay)
    for group, places in ((0, slice(0, N)), (128, slice(0, N))):
        codes, scales, _ = mla.residual_norm_fp8(x, r, w, group=group, rms_eps=1e-6)
        c = codes.float()
        for row in (0, 4, 6):
            assert (c[row] == 0).all() and (scales[row] == 1).all()
        assert torch.isnan(c[1]).all() and torch.isnan(scales[1]).all()              # (the norm of the row is NaN)
        broken = slice(256, 384) if group else places
        assert torch.isnan(c[2, broken]).all() and torch.isnan(scales[2, 2 if group else 0])
        # 1e-38 / 1e-3 = 1e-35 in every place: the largest code everywhere, the scale 1e-35 / 448
        assert (c[3] == 448).all() and ((scales[3].double() / (float(x[3, 0]) * 1e3 / 448) - 1).abs() <= 1e-3).all()
        y = OC.residual_norm(x[5:6], None, w, 1e-6)[0]
        assert (c[5, :128] == 448).all() and (c[5, 128:] == 0).all()
        assert abs(float(scales[5, 0]) * 448 / float(y[0, 0]) - 1) <= 1e-5


def test_captured_layer_boundary():
    x, r, w = normal(40, 7168, seed=15), normal(40, 7168, seed=16), normal(7168, seed=17)
    q, positions = normal(40, 128, 64, seed=18), torch.arange(40, dtype=torch.int32, device="cuda")
    table = mla.rope_table()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            a = mla.residual_norm(x, r, w)
            b = mla.residual_norm_fp8(x, r, w)
            c = mla.rotate(q, positions, table=table)
    x.mul_(2)
    q.mul_(-1)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    for got, want in zip((*a, *b, c), (*mla.residual_norm(x, r, w), *mla.residual_norm_fp8(x, r, w),
                                       mla.rotate(q, positions, table=table))):
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


def test_a_large_array():
    """Rows past 2^31 elements."""
    T = 300000                                              # 2.15e9 values
    x = torch.zeros(T, 7168, dtype=torch.bfloat16, device="cuda")
    x[-3:] = normal(3, 7168, seed=19)
    w = normal(7168, seed=20)
    out, _ = mla.residual_norm(x, None, w)
    small, _ = mla.residual_norm(x[-3:].clone(), None, w)
    assert torch.equal(out[-3:], small) and (out[:5] == 0).all()
    del out
    q = x.view(T, 56, 128)
    positions = torch.full((T,), 1234, dtype=torch.int32, device="cuda")
    table = mla.rope_table_scaled(dims=128)
    y = mla.rotate(q, positions, table=table, layout="half")
    assert torch.equal(y[-3:], mla.rotate(q[-3:].clone(), positions[-3:], table=table, layout="half"))


def test_refusals():
    x, w = normal(4, 64, seed=21), normal(64, seed=22)
    for bad in (lambda: mla.residual_norm(x[:, :60], None, w[:60]), lambda: mla.residual_norm(x, x[:3], w),
                lambda: mla.residual_norm(x, None, w[:32]), lambda: mla.residual_norm(x, None, w, residual_out=x.clone()),
                lambda: mla.residual_norm(x.cpu(), None, w), lambda: mla.residual_norm(x.t(), None, w),
                lambda: mla.residual_norm(x[:0], None, w), lambda: mla.residual_norm_fp8(x, None, w, group=64),
                lambda: mla.residual_norm_fp8(x, x, w, scales=torch.empty(4, 2, device="cuda")),
                lambda: mla.residual_norm(x, None, w, out=torch.empty(4, 32, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mla.residual_norm(x.float(), None, w), lambda: mla.residual_norm(x, x.half(), w),
                lambda: mla.residual_norm_fp8(x, x, w, codes=torch.empty(4, 64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(TypeError):
            bad()
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(mla.MLAError):
            mla.residual_norm(x, None, w, rms_eps=eps)
    q, pos, table = normal(4, 8, 64, seed=23), torch.zeros(4, dtype=torch.int32, device="cuda"), mla.rope_table()
    for bad in (lambda: mla.rotate(q[..., :48], pos, table=table), lambda: mla.rotate(q, pos[:3], table=table),
                lambda: mla.rotate(q, pos, table=table[:32]), lambda: mla.rotate(q, pos, table=table, layout="other"),
                lambda: mla.rotate(q, pos, table=table, out=q[:3]), lambda: mla.rotate(q[0], pos, table=table),
                lambda: mla.rotate(q.transpose(1, 2), pos, table=table), lambda: mla.rope_table_scaled(dims=48)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        mla.rotate(q, pos.long(), table=table)
    for kw in (dict(rope_base=1.0), dict(factor=0.5), dict(factor=float("nan")), dict(original_positions=0), dict(beta_slow=0.0),
               dict(beta_fast=0.5), dict(rope_base=float("inf"))):
        with pytest.raises(mla.MLAError):
            mla.rope_table_scaled(**kw)
    with pytest.raises(mla.MLAError):
        mla.rotate(q, pos, table=table, magnitude=float("nan"))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_a_chunk_through_the_layer(fp8):
    """Append, rotate, attention, output projection and norm as they run together, two chunks of a prompt after one
    another; each step against 64 bits from what it was given."""
    T, hidden = 150, 1024
    w_uk, w_uv = normal(128, 128, 512, seed=24, std=512 ** -0.5), normal(128, 128, 512, seed=25, std=512 ** -0.5)
    w_o, gamma, weight = normal(hidden, 16384, seed=26, std=1 / 128), normal(512, seed=27), normal(hidden, seed=28)
    table, rate = mla.rope_table_scaled(factor=40.0), OC.rates(64, factor=40.0)
    pages = 12
    cache = torch.zeros(pages, 64, 656, dtype=torch.uint8, device="cuda") if fp8 else \
        torch.full((pages, 64, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    block_table = torch.tensor([[7, 2, 9, 0, 5], [3, 11, 1, 4, 8]], dtype=torch.int32, device="cuda")
    lens = [0, 0]
    residual = normal(T, hidden, seed=29)
    for step, counts in enumerate(([100, 50], [30, 120])):
        lens = [a + b for a, b in zip(lens, counts)]
        off = torch.tensor([0, counts[0], T], dtype=torch.int32, device="cuda")
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        pos = torch.cat([torch.arange(L - n, L) for n, L in zip(counts, lens)]).to(torch.int32).cuda()
        kv, q = normal(T, 576, seed=30 + step), normal(T, 128, 192, seed=40 + step)
        raw = q.clone()
        append = mla.cache_append_fp8 if fp8 else mla.cache_append
        st = append(kv[:, :512], kv[:, 512:], gamma, cache, block_table, sl, off, table=table)
        mla.rotate(q[..., 128:], pos, table=table, out=q[..., 128:])
        check_rotated(q[..., 128:], raw[..., 128:], pos, rate, False)
        p = mla.chunk_plan(sl, off, tokens=T, max_pages_per_seq=5, kv_tokens=sum(-(-L // 64) * 64 for L in lens))
        o = (mla.chunk_attend_fp8 if fp8 else mla.chunk_attend)(p, q[..., :128], q[..., 128:], w_uk, w_uv, cache, block_table)
        assert mla.check(p) == 0 and int(st.item()) == 0
        ref = OC.chunk_attend(q, w_uk, w_uv, cache, block_table, lens, off.tolist(), scale=mla.DEFAULT_SCALE)[0]
        rows = (o.double() - ref).norm(dim=-1) / ref.norm(dim=-1)
        # keys of size |gamma|: scores of a deviation above 1, their error 0.82 BF / sqrt(3) of the deviation
        assert rows.max() <= 3e-2 and (o.double() - ref).norm() <= 8e-3 * ref.norm()
        out = mla.epilog_oproj(o, w_o)
        want = o.view(T, 16384).double() @ w_o.double().T
        assert ((out.double() - want).abs() <= BF * want.abs() + 16384 * 2.0 ** -24 * (o.view(T, 16384).double().abs() @ w_o.double().abs().T)).all()
        y, kept = mla.residual_norm(out, residual, weight)
        check_norm(out, residual, weight, y, kept, 1e-6)
        codes, scales, kept8 = mla.residual_norm_fp8(out, residual, weight)
        assert torch.equal(kept8, kept)
        y8 = codes.double() * scales.double().repeat_interleave(128, 1)
        exact = OC.residual_norm(out, residual, weight, 1e-6)[0]
        assert ((y8 - exact).abs() <= 2.0 ** -4 * exact.abs() + scales.double().repeat_interleave(128, 1) * 2.0 ** -10 + 1e-4 * exact.abs()).all()
        residual = kept


def test_calls_marshalled_in_python_are_the_same(monkeypatch):
    import chunk_util as CU
    import mla_decode_attention_02_gb300._binding as binding
    c = CU.case([70, 9], [200, 150], seed=50)
    x, r, w = normal(7, 1032, seed=51), normal(7, 1032, seed=52), normal(1032, seed=53)
    q, positions, table = normal(7, 5, 64, seed=54), torch.arange(7, dtype=torch.int32, device="cuda"), mla.rope_table()
    s = torch.cuda.Stream()

    def all_of_them(**kw):
        p = mla.chunk_plan(c["seq_lens"], c["offsets"], tokens=c["T"], max_pages_per_seq=c["block_table"].shape[1],
                           kv_tokens=c["kv_tokens"], **kw)
        lse = torch.empty(c["T"], 128, device="cuda")
        return [mla.rotate(q, positions, table=table, layout="half", **kw),
                mla.rotate(q, positions, table=table, inverse=True, magnitude=2, out=torch.empty_like(q), **kw),
                *mla.residual_norm(x, r, w, **kw), mla.residual_norm(x, None, w, **kw)[0], *mla.residual_norm_fp8(x, r, w, **kw),
                *mla.residual_norm_fp8(x, r, w, group=0, **kw), *mla.residual_norm_fp8(x, None, w, **kw)[:2],
                mla.chunk_attend(p, c["q"][..., :128], c["q"][..., 128:], c["w_uk"], c["w_uv"], c["cache"], c["block_table"],
                                 lse=lse, **kw), lse, mla.rope_table_scaled(factor=8.0, **kw)]

    native = all_of_them()
    s.wait_stream(torch.cuda.current_stream())
    on_stream = all_of_them(stream=s)
    s.synchronize()
    monkeypatch.setattr(binding, "_host", binding._PythonOnly)
    python = all_of_them()
    assert len(native) == len(python) == len(on_stream)
    for a, b, d in zip(native, python, on_stream):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(a.view(torch.uint8), d.view(torch.uint8))
