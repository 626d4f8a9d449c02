"""Rotary positions and the cache appends on the GPU against the fp64 oracle.

A rotated value m (a cos t - b sin t) computed in fp32 is off by at most
ROT * m * (|a| + |b|): the angle by pi 2^-25 (the phase rounded to fp32), cos
and sin by another 2^-23, the factor, products and sum by 2^-24 each, under
2^-21 in all.  Where such a value is then rounded to codes, the stored code
must be the code of some value within that distance; what is not rotated is
held to the code itself."""
import numpy as np
import pytest
import torch

from oracle import msa_oracle as O

pytestmark = pytest.mark.gpu
ROT = 2.0 ** -21
BF16 = 2.0 ** -8


def _msa():
    from block_sparse_long_proxy_gb300 import msa
    return msa


def _rope(rot, layout="half", **scaling):
    return _msa().Rope(rot, layout=layout, **scaling)


def _partner_sum(x, rot, layout):
    """|a| + |b| of each value's pair; 0 behind the rotated dims."""
    a = np.abs(x)
    out = np.zeros_like(a)
    lo, hi = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    out[..., lo] = out[..., hi] = a[..., lo] + a[..., hi]
    return out


def _f64(t):
    return t.detach().double().cpu().numpy()


# -------------------------------------------------------------------- rope --

ROPES = [
    # rows, heads, head_dim, rotary_dim, layout, dtype, inverse, row gap, first position, scaling
    (1, 1, 16, 16, "half", "bf16", False, 0, 0, {}),
    (1, 64, 128, 128, "half", "bf16", False, 0, 131071, {}),
    (3, 5, 128, 128, "interleaved", "fp32", True, 8, 5, {}),
    (77, 3, 48, 32, "half", "fp32", False, 4, 2 ** 31 - 100, {}),
    (200, 7, 64, 48, "interleaved", "bf16", True, 24, -150, dict(scaling="linear", factor=4.0)),
    (513, 9, 80, 16, "half", "bf16", False, 0, 99, dict(scaling="ntk", factor=8.0)),
    (1000, 40, 128, 64, "half", "fp32", True, 0, 10 ** 6, dict(scaling="yarn", factor=16.0, original_len=8192)),
    (2500, 16, 256, 256, "interleaved", "bf16", False, 512, 40000, dict(base=5e5)),
    (5000, 33, 32, 32, "half", "bf16", True, 0, 7, {}),
]


@pytest.mark.parametrize("n, heads, d, rot, layout, dtype, inverse, gap, first, scaling", ROPES)
def test_rope_apply(cuda_dev, n, heads, d, rot, layout, dtype, inverse, gap, first, scaling):
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device=cuda_dev).manual_seed(n)
    wide = torch.randn((n, heads * d + gap), generator=gen, device=cuda_dev).to(t)
    x = wide[:, :heads * d].unflatten(1, (heads, d))
    pos = torch.arange(first, first + n, device=cuda_dev).to(torch.int32)
    got = _rope(rot, layout, **scaling).apply(x, pos, inverse=inverse)
    xs = _f64(x)
    ref = O.rope(xs, pos.cpu().numpy(), rot, layout, inverse, **scaling)
    m = O.rope_freqs(rot, **scaling)[1]
    tol = ROT * m * _partner_sum(xs, rot, layout)
    if dtype == "bf16":
        tol = tol + BF16 * (np.abs(ref) + tol)
    assert (np.abs(_f64(got) - ref) <= tol).all()
    assert np.array_equal(_f64(got)[..., rot:], xs[..., rot:])


def test_rope_in_place_slices_and_streams(cuda_dev):
    """In place; from one slice of a projection's rows to another; on a side
    stream; captured in a graph and replayed over new inputs."""
    rope = _rope(32)
    gen = torch.Generator(device=cuda_dev).manual_seed(0)
    wide = torch.randn((300, 3 * 4 * 64), generator=gen, device=cuda_dev).to(torch.bfloat16)
    pos = torch.randint(0, 100000, (300,), generator=gen, device=cuda_dev, dtype=torch.int32)
    q, k, v = (wide[:, i * 256:(i + 1) * 256].unflatten(1, (4, 64)) for i in range(3))
    want = rope.apply(q.clone(), pos)
    v0, q0 = v.clone(), q.clone()
    rope.apply(q, pos, out=k)
    assert torch.equal(k, want) and torch.equal(q, q0) and torch.equal(v, v0)
    rope.apply(q, pos, out=q)
    assert torch.equal(q, want) and torch.equal(v, v0)
    with pytest.raises(_msa().MsaError):
        rope.apply(q[:, :2], pos, out=q[:, 1:3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rope.apply(q0, pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out, src = torch.empty_like(q0), q0.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope.apply(src, pos, out=out)
    src.copy_(v0)
    graph.replay()
    assert torch.equal(out, rope.apply(v0, pos))
    assert rope.apply(q0[:0], pos[:0]).shape == (0, 4, 64)


@pytest.mark.parametrize("layout, inverse, scaling", [("half", False, {}), ("interleaved", True, {}),
                                                      ("half", True, dict(scaling="yarn", factor=8.0, original_len=4096))])
def test_rope_has_the_bits_of_elementwise_arithmetic(cuda_dev, layout, inverse, scaling):
    """cos and sin from fp64, products and sums rounded in fp32: equal but where a
    cosine (1 of 200) or a sine (1 of 40) is the other neighbour, and there by the
    rounding of a value and of two products."""
    n, rot = 4000, 64
    gen = torch.Generator(device=cuda_dev).manual_seed(4)
    x = torch.randn((n, 2, rot), generator=gen, device=cuda_dev)
    pos = torch.randint(0, 200000, (n,), generator=gen, device=cuda_dev, dtype=torch.int32)
    got = _rope(rot, layout, **scaling).apply(x, pos, inverse=inverse)
    f, m = O.rope_freqs(rot, **scaling)
    t = np.outer(pos.cpu().numpy(), f / (2 * np.pi))
    t = (t - np.floor(t)) * 2 * np.pi
    c, s = (torch.from_numpy((y * m).astype(np.float32)).to(cuda_dev)[:, None] for y in (np.cos(t), np.sin(t)))
    s = -s if inverse else s
    a, b = (x[..., :32], x[..., 32:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])
    p, q = a * c - b * s, b * c + a * s
    want = torch.cat((p, q), -1) if layout == "half" else torch.stack((p, q), -1).flatten(-2)
    assert (got != want).float().mean() <= 0.05 and (got - want).abs().max() <= 1e-6 * 5


def test_rope_inverse_is_the_gradient(cuda_dev):
    """<rope(x), y> = <x, inverse(y)>, and central differences of it."""
    rope = _rope(64, "interleaved", scaling="yarn", factor=4.0, original_len=1024)
    gen = torch.Generator(device=cuda_dev).manual_seed(2)
    x, y = (torch.randn((50, 2, 64), generator=gen, device=cuda_dev) for _ in range(2))
    pos = torch.arange(50, device=cuda_dev, dtype=torch.int32) * 401
    dx = rope.apply(y, pos, inverse=True)
    lhs, rhs = (rope.apply(x, pos) * y).double().sum(), (x * dx).double().sum()
    # every product is off by ROT * m * (|a| + |b|) * |other| at most; m < 1.2
    room = 1.2 * ROT * 4 * float(((x.abs() + 4) * (y.abs() + 4)).sum()) / 4
    assert abs(float(lhs - rhs)) <= room
    for r, h, i in ((0, 0, 0), (7, 1, 13), (49, 0, 63)):
        e = torch.zeros_like(x)
        e[r, h, i] = 0.5
        diff = ((rope.apply(x + e, pos) - rope.apply(x - e, pos)) * y).double().sum()
        assert abs(float(diff - dx[r, h, i])) <= 1e-4     # fp32 values of order 1..5: 2^-21 * 5 * 5 * 4 terms


# ----------------------------------------------------------------- appends --

LENS = {
    "one token": ([1], [1]),
    "one token behind 127": ([1], [128]),
    "first token of a page": ([1], [129]),
    "decode batch": ([1] * 7, [1, 128, 129, 5000, 77, 1024, 300]),
    "chunks": ([300, 0, 77, 128, 129], [300, 90, 1000, 128, 500]),
    "long": ([4000], [4321]),
}


def _setup(qo, kv, hkv, d, dp, kind, dev, seed, extra=2):
    nb = [(k + 127) // 128 for k in kv]
    gen = torch.Generator(device=dev).manual_seed(seed)
    p = sum(nb) + extra
    table = torch.randperm(p, generator=gen, device=dev)[:sum(nb)].to(torch.int32)
    plan = _msa().Plan(qo, kv, hkv, hkv, hkv, d, dp, 1, p, kv_dtype=kind)
    return plan, table, gen, p


def _fresh_codes(shape, gen, dev):
    """Codes of values up to 448, no NaN among them."""
    return torch.randn(shape, generator=gen, device=dev).mul(120).clamp(-448, 448).to(torch.float8_e4m3fn)


def _codes_between(got, x, delta, by):
    """Every stored code is that of a value within delta of x, over by."""
    val = O.e4m3_to_f64(got)
    lo, hi = O.e4m3_to_f64(O.to_e4m3((x - delta) / by)), O.e4m3_to_f64(O.to_e4m3((x + delta) / by))
    assert (val >= lo).all() and (val <= hi).all()


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("kind, d, rot, layout", [("bf16", 64, 64, "half"), ("bf16", 128, 32, "interleaved"),
                                                  ("e4m3", 128, 128, "half"), ("e4m3", 64, 16, "interleaved"),
                                                  ("e4m3_block", 128, 128, "half"),
                                                  ("e4m3_block", 128, 96, "interleaved"), ("e4m3_block", 64, 0, "half")])
def test_kv_append(cuda_dev, lens, kind, d, rot, layout):
    qo, kv = LENS[lens]
    hkv, rows = 3, sum(qo)
    plan, table, gen, p = _setup(qo, kv, hkv, d, 32, kind, cuda_dev, 5)
    wide = (torch.randn((rows, 2 * hkv * d + 8), generator=gen, device=cuda_dev)
            * torch.exp(torch.randn((rows, 1), generator=gen, device=cuda_dev))).to(torch.bfloat16)
    k, v = (wide[:, i * hkv * d:(i + 1) * hkv * d].unflatten(1, (hkv, d)) for i in range(2))
    shape = (p, hkv, 128, d)
    if kind == "bf16":
        pages = [torch.randn(shape, generator=gen, device=cuda_dev).to(torch.bfloat16) for _ in range(2)]
        scales = [None, None]
    else:
        pages = [_fresh_codes(shape, gen, cuda_dev) for _ in range(2)]
        if kind == "e4m3":
            scales = [torch.rand(hkv, generator=gen, device=cuda_dev) * 0.02 + 0.002 for _ in range(2)]
        else:  # pages whose first slot is written start anew, whatever they held; others hold a power of two
            scales = [torch.exp2(torch.randint(-12, 0, (p, hkv), generator=gen, device=cuda_dev).float())
                      for _ in range(2)]
    before = [t.clone() for t in pages]
    old_scales = [None if s is None else _f64(s) for s in scales]
    rope = _rope(rot, layout) if rot else None
    off = 1000
    key_pos = np.concatenate([np.arange(b - a, b) for a, b in zip(qo, kv)])
    positions = torch.from_numpy((key_pos + off).astype(np.int32)).to(cuda_dev)
    plan.kv_append(k, v, *pages, table, k_scale=scales[0], v_scale=scales[1], rope=rope, positions=positions)
    plan.check_errors()
    for x, t, b, s, old, turned in ((k, pages[0], before[0], scales[0], old_scales[0], rot > 0),
                                    (v, pages[1], before[1], scales[1], old_scales[1], False)):
        xs = _f64(x)
        ref = O.rope(xs, key_pos + off, rot, layout) if turned else xs
        delta = ROT * _partner_sum(xs, rot, layout) if turned else np.zeros_like(xs)
        if kind == "bf16":
            want, _ = O.kv_append(ref, _f64(b), table.cpu().numpy(), qo, kv, kind)
            dl, _ = O.kv_append(delta, np.zeros(shape), table.cpu().numpy(), qo, kv, kind)
            tol = dl + (BF16 * (np.abs(want) + dl) if turned else 0.0) * (dl > 0)
            assert (np.abs(_f64(t) - want) <= tol).all()
            continue
        got, raw = t.view(torch.uint8).cpu().numpy(), b.view(torch.uint8).cpu().numpy()
        if kind == "e4m3":
            by = _f64(s)[None, :, None]
            delta = delta + np.abs(ref) * 2.0 ** -24              # the quotient is rounded once before the code
            lo, _ = O.kv_append(ref, raw, table.cpu().numpy(), qo, kv, kind, _f64(s))
            rows_ref = dict(lo=ref - delta, hi=ref + delta)
            bound = {n: O.kv_append(r, raw, table.cpu().numpy(), qo, kv, kind, _f64(s))[0] for n, r in rows_ref.items()}
            g = O.e4m3_to_f64(got)
            assert (g >= np.minimum(O.e4m3_to_f64(bound["lo"]), O.e4m3_to_f64(bound["hi"]))).all()
            assert (g <= np.maximum(O.e4m3_to_f64(bound["lo"]), O.e4m3_to_f64(bound["hi"]))).all()
            assert by.shape == (1, hkv, 1) and lo.shape == got.shape
            continue
        want, want_s = O.kv_append(ref, raw, table.cpu().numpy(), qo, kv, kind, old)
        if not turned:
            assert np.array_equal(_f64(s), want_s) and np.array_equal(got, want)
            continue
        # the scale from the oracle: a page's largest value may lie within delta of a border only here
        same = _f64(s) == want_s
        assert same.mean() > 0.99
        g, w = O.e4m3_to_f64(got), O.e4m3_to_f64(want)
        d_at, _ = O.kv_append(delta, np.zeros(shape), table.cpu().numpy(), qo, kv, "bf16")
        x_at, _ = O.kv_append(ref, np.full(shape, np.nan), table.cpu().numpy(), qo, kv, "bf16")
        new = ~np.isnan(x_at) & same[:, :, None, None]
        assert np.array_equal(g[np.isnan(x_at) & same[:, :, None, None]], w[np.isnan(x_at) & same[:, :, None, None]])
        by = np.broadcast_to(_f64(s)[:, :, None, None], shape)
        _codes_between(got[new], x_at[new], d_at[new], by[new])


def test_kv_append_row_by_row(cuda_dev):
    """A page filled token by token: the scale follows the largest value, and
    the codes are those of the oracle's same steps."""
    d, steps = 128, 130
    gen = torch.Generator(device=cuda_dev).manual_seed(9)
    rows = (torch.randn((steps, 1, d), generator=gen, device=cuda_dev)
            * torch.logspace(-3, 2, steps, device=cuda_dev)[torch.randperm(steps, generator=gen, device=cuda_dev), None,
                                                            None]).to(torch.bfloat16)
    pages = [torch.full((3, 1, 128, d), 0x7F, dtype=torch.uint8, device=cuda_dev).view(torch.float8_e4m3fn)
             for _ in range(2)]
    scale = [torch.full((3, 1), float("nan"), device=cuda_dev) for _ in range(2)]
    table = torch.tensor([2, 0], dtype=torch.int32, device=cuda_dev)
    want, ws = np.full((3, 1, 128, d), 0x7F, np.uint8), np.full((3, 1), np.nan)
    for i in range(steps):
        plan = _msa().Plan([1], [i + 1], 1, 1, 1, d, 32, 1, 3, kv_dtype="e4m3_block")
        x = rows[i:i + 1]
        plan.kv_append(x, x, *pages, table[:plan.n_page_entries], k_scale=scale[0], v_scale=scale[1])
        plan.check_errors()
        want, ws = O.kv_append(_f64(x), want, table.cpu().numpy(), [1], [i + 1], "e4m3_block", ws)
    for t, s in zip(pages, scale):
        assert np.array_equal(t.view(torch.uint8).cpu().numpy(), want)
        assert np.array_equal(_f64(s), ws, equal_nan=True)


def test_kv_append_extremes(cuda_dev):
    """Zero rows get the least scale, infinities saturate without setting the
    scale, values past 448 * 2^40 saturate, NaN stays in its slot; another
    writer's scale is rounded up to a power of two."""
    plan, table, gen, p = _setup([5], [10], 1, 64, 32, "e4m3_block", cuda_dev, 1)
    inf, nan = float("inf"), float("nan")
    k = torch.ones((5, 1, 64), device=cuda_dev)
    k[1, 0, 3], k[2, 0, 4], k[3, 0, 5] = inf, -inf, nan
    v = torch.zeros((5, 1, 64), device=cuda_dev)
    pages = [_fresh_codes((p, 1, 128, 64), gen, cuda_dev) for _ in range(2)]
    before = [t.view(torch.uint8).clone() for t in pages]
    scales = [torch.full((p, 1), 0.011, device=cuda_dev) for _ in range(2)]
    plan.kv_append(k.bfloat16(), v.bfloat16(), *pages, table, k_scale=scales[0], v_scale=scales[1])
    plan.check_errors()
    page = int(table[0])
    s = 2.0 ** -6                                       # 0.011 rounded up
    assert float(scales[0][page]) == s and float(scales[1][page]) == s
    old = O.to_e4m3(O.e4m3_to_f64(before[0][page, 0, :5].cpu().numpy()) * float(np.float32(0.011)) / s)
    assert np.array_equal(pages[0].view(torch.uint8)[page, 0, :5].cpu().numpy(), old)
    got = pages[0][page, 0, 5:10].float().cpu().numpy() * s
    assert got[1, 3] == 448 * s and got[2, 4] == -448 * s and np.isnan(got[3, 5])
    got[1, 3] = got[2, 4] = got[3, 5] = 1.0
    assert (got == 1.0).all() and (pages[1][page, 0, 5:10].float() == 0).all()
    plan2, table2, gen, p = _setup([2], [2], 1, 64, 32, "e4m3_block", cuda_dev, 1)
    k = torch.full((2, 1, 64), 1e30, device=cuda_dev).bfloat16()
    plan2.kv_append(k, torch.zeros_like(k), *pages, table2, k_scale=scales[0], v_scale=scales[1])
    assert float(scales[0][int(table2[0])]) == 2.0 ** 40 and float(scales[1][int(table2[0])]) == 2.0 ** -40
    assert (pages[0][int(table2[0]), 0, :2].float() == 448).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3_block"])
def test_kv_append_bad_pages_and_scales(cuda_dev, kind):
    """A page outside the pool drops its rows and is reported; so is a partly
    filled page whose scale was never written, whose old slots stay."""
    msa = _msa()
    qo, kv = [200, 3], [300, 9]
    plan, table, gen, p = _setup(qo, kv, 2, 64, 32, kind, cuda_dev, 3)
    k = torch.randn((203, 2, 64), generator=gen, device=cuda_dev).bfloat16()
    if kind == "bf16":
        pages, scales = [torch.zeros((p, 2, 128, 64), dtype=torch.bfloat16, device=cuda_dev) for _ in range(2)], [None] * 2
    else:
        pages = [_fresh_codes((p, 2, 128, 64), gen, cuda_dev) for _ in range(2)]
        scales = [torch.full((p, 2), 2.0 ** -5, device=cuda_dev) for _ in range(2)]
    for bad in (-1, p, 2 ** 31 - 1):
        t2 = table.clone()
        t2[1] = bad
        before = [t.clone() for t in pages]
        plan.kv_append(k, k, *pages, t2, k_scale=scales[0], v_scale=scales[1])
        with pytest.raises(msa.MsaError) as e:
            plan.check_errors()
        assert e.value.status == 6
        assert torch.equal(pages[0].view(torch.uint8)[table[1].long()], before[0].view(torch.uint8)[table[1].long()])
    if kind == "bf16":
        return
    for s in (0.0, float("nan"), -1.0, float("inf"), 2.0 ** 41):
        scales[0].fill_(s)
        before = pages[0].view(torch.uint8).clone()
        plan.kv_append(k, k, *pages, table, k_scale=scales[0], v_scale=scales[1])
        with pytest.raises(msa.MsaError) as e:
            plan.check_errors()
        assert e.value.status == 6
        first = int(table[0])                            # rows 100.. behind 100 old ones
        assert torch.equal(pages[0].view(torch.uint8)[first, :, :100], before[first, :, :100])
        assert torch.isfinite(scales[0][table.long()]).all()


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dp, rot, layout", [(64, 64, "half"), (64, 48, "half"), (32, 16, "interleaved"), (32, 0, "half")])
def test_pk_append(cuda_dev, lens, dp, rot, layout):
    qo, kv = LENS[lens]
    rows = sum(qo)
    plan, table, gen, p = _setup(qo, kv, 1, 64, dp, "bf16", cuda_dev, 7)
    pk = torch.randn((rows, 1, dp), generator=gen, device=cuda_dev).mul(2).bfloat16()
    pk[0] = 0.0
    if rows > 2:
        pk[1] *= 1e-6       # block scales round to 0
        pk[2] *= 1e4        # block scales saturate
    g, s8 = 8.0 / (448 * 6), 0.013
    pool = (p, 1, 128)
    bf = torch.randn(pool + (dp,), generator=gen, device=cuda_dev).bfloat16()
    e8 = _fresh_codes(pool + (dp,), gen, cuda_dev)
    codes = torch.randint(0, 256, pool + (dp // 2,), generator=gen, device=cuda_dev).to(torch.uint8)
    bs = _fresh_codes(pool + (dp // 16,), gen, cuda_dev)
    before = [t.clone() for t in (bf, e8, codes, bs)]
    gs, ss = (torch.full((1,), x, device=cuda_dev) for x in (g, s8))
    rope = _rope(rot, layout) if rot else None
    plan.pk_append(pk, table, pk_pages=bf, pk_pages_e4m3=e8, pk_scale=ss, pk_codes=codes, pk_block_scales=bs,
                   pk_global_scale=gs, rope=rope)
    plan.check_errors()
    pos = np.concatenate([np.arange(b - a, b) for a, b in zip(qo, kv)])
    x = _f64(pk)
    ref = O.rope(x, pos, rot, layout) if rot else x
    delta = ROT * _partner_sum(x, rot, layout) if rot else np.zeros_like(x)
    at = [int(table[e]) for e in np.concatenate([[b + q // 128 for q in range(k - n, k)] for b, n, k in
                                                 zip(O.kv_indptr(kv)[:-1], qo, kv) if n]).astype(int)]
    slot = pos % 128
    untouched = np.ones((p, 128), bool)
    untouched[at, slot] = False
    for t, b in zip((bf, e8, codes, bs), before):
        t, b = (y.view(torch.uint8).cpu().numpy()[:, 0] for y in (t, b))
        assert np.array_equal(t[untouched], b[untouched])
    got = _f64(bf)[at, 0, slot]
    assert (np.abs(got - ref[:, 0]) <= (delta + (BF16 * (np.abs(ref) + delta)) * (delta > 0))[:, 0]).all()
    _codes_between(e8.view(torch.uint8).cpu().numpy()[at, 0, slot], ref[:, 0],
                   (delta + np.abs(ref) * 2.0 ** -24)[:, 0], float(ss))
    got_bs = bs.view(torch.uint8).cpu().numpy()[at, 0, slot]
    got_c = codes.cpu().numpy()[at, 0, slot]
    want_c, want_bs = O.to_nvfp4(ref[:, 0], float(gs))
    if not rot:
        assert np.array_equal(got_bs, want_bs) and np.array_equal(got_c, want_c)
        return
    blocks, dl = (y[:, 0].reshape(rows, -1, 16) for y in (ref, delta))
    lo, hi = (O.to_e4m3(np.maximum(np.abs(blocks).max(-1) + sg * dl.max(-1), 0) / (6 * float(gs))) for sg in (-1, 1))
    assert ((got_bs >= lo) & (got_bs <= hi)).all()
    val = O.nvfp4_to_f64(got_c, got_bs, float(gs)).reshape(rows, -1, 16)
    by = (O.e4m3_to_f64(got_bs) * float(gs))[..., None]
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6]) * by[..., None]
    best = np.abs(np.abs(blocks)[..., None] - grid).min(-1)
    assert (np.abs(val - blocks) <= best + 2 * dl + 1e-15).all()


@pytest.mark.parametrize("lens", LENS)
def test_append_bwd(cuda_dev, lens):
    """Rows of the gradient pages, K's and the proxy's rotated back: the
    transpose of the append."""
    qo, kv = LENS[lens]
    rows, hkv, d, dp = sum(qo), 3, 128, 64
    plan, table, gen, p = _setup(qo, kv, hkv, d, dp, "bf16", cuda_dev, 11)
    dk, dv = (torch.randn((p, hkv, 128, d), generator=gen, device=cuda_dev) for _ in range(2))
    dpk = torch.randn((p, 1, 128, dp), generator=gen, device=cuda_dev)
    k_rope, pk_rope = _rope(96, "half"), _rope(32, "interleaved", scaling="yarn", factor=2.0, original_len=4096)
    got = plan.append_bwd(table, dk_pages=dk, dv_pages=dv, dpk_pages=dpk, k_rope=k_rope, pk_rope=pk_rope)
    plan.check_errors()
    pos = np.concatenate([np.arange(b - a, b) for a, b in zip(qo, kv)])
    entry = np.concatenate([[b + q // 128 for q in range(k - n, k)] for b, n, k in
                            zip(O.kv_indptr(kv)[:-1], qo, kv) if n]).astype(int)
    page = table.cpu().numpy()[entry]
    for t, g, rot, layout, kw in ((dk, got[0], 96, "half", {}), (dv, got[1], 0, "half", {}),
                                  (dpk, got[2], 32, "interleaved", dict(scaling="yarn", factor=2.0, original_len=4096))):
        x = _f64(t)[page, :, pos % 128]
        if not rot:
            assert np.array_equal(_f64(g), x)
            continue
        tol = ROT * 1.2 * _partner_sum(x, rot, layout)
        assert (np.abs(_f64(g) - O.rope(x, pos, rot, layout, inverse=True, **kw)) <= tol).all()
    # one of the three alone, and a page outside the pool: its rows are zero
    only = plan.append_bwd(table, dv_pages=dv)
    assert only[0] is None and only[2] is None and torch.equal(only[1], got[1])
    bad = table.clone()
    bad[int(entry[0])] = p
    rows_of = torch.from_numpy(entry == entry[0]).to(cuda_dev)
    got2 = plan.append_bwd(bad, dk_pages=dk, k_rope=k_rope)[0]
    with pytest.raises(_msa().MsaError) as e:
        plan.check_errors()
    assert e.value.status == 6
    assert (got2[rows_of] == 0).all() and torch.equal(got2[~rows_of], got[0][~rows_of])


@pytest.mark.parametrize("call", ["bf16", "proxy", "bwd"])
def test_append_pages_beyond_4_gib(cuda_dev, call):
    """The last pages of pools of more than 2^32 bytes, bit for bit as on small
    pools; the first pages stay as they were."""
    from block_sparse_long_proxy_gb300 import msa
    hkv, n = 8, {"bf16": 17000, "proxy": 263000, "bwd": 8500}[call]
    gen = torch.Generator(device=cuda_dev).manual_seed(5)
    table = torch.tensor([4, 1, 0, 3], dtype=torch.int32, device=cuda_dev)   # of the last five pages
    rope = msa.Rope(64)
    got = []
    for pages in (5, n):
        plan = msa.Plan([200, 1], [300, 128], 8, hkv, hkv, 128, 64, 2, pages)
        ids = table + (pages - 5)
        gen.manual_seed(6)
        rows = lambda h, d: torch.randn((201, h, d), generator=gen, device=cuda_dev).bfloat16()  # noqa: E731
        zeros = lambda h, d, t: torch.zeros((pages, h, 128, d), dtype=t, device=cuda_dev)  # noqa: E731
        if call == "bf16":
            pools = [zeros(hkv, 128, torch.bfloat16) for _ in "kv"]
            plan.kv_append(rows(hkv, 128), rows(hkv, 128), *pools, ids, rope=rope)
        elif call == "proxy":
            f8 = lambda d: zeros(1, d, torch.uint8).view(torch.float8_e4m3fn)  # noqa: E731
            one = torch.full((1,), 0.01, device=cuda_dev)
            pools = [zeros(1, 64, torch.bfloat16), f8(64), zeros(1, 32, torch.uint8), f8(4)]
            plan.pk_append(rows(1, 64), ids, pk_pages=pools[0], pk_pages_e4m3=pools[1], pk_scale=one, pk_codes=pools[2],
                           pk_block_scales=pools[3], pk_global_scale=one, rope=rope)
        else:
            pools = [zeros(hkv, 128, torch.float32) for _ in "kv"]
            for x in pools:
                x[-5:] = torch.randn((5, hkv, 128, 128), generator=gen, device=cuda_dev)
            got.append(plan.append_bwd(ids, dk_pages=pools[0], dv_pages=pools[1], k_rope=rope)[:2])
        plan.check_errors()
        if call != "bwd":
            got.append([x[-5:].view(torch.uint8).clone() for x in pools])
            assert all(x.any().item() for x in got[-1])
            if pages > 5:
                assert not any(x.view(torch.uint8)[:5].any().item() for x in pools)
        del pools
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_append_refusals(cuda_dev):
    msa = _msa()
    plan, table, gen, p = _setup([4], [4], 2, 64, 32, "e4m3_block", cuda_dev, 0)
    k = torch.zeros((4, 2, 64), device=cuda_dev).bfloat16()
    pages = [torch.zeros((p, 2, 128, 64), device=cuda_dev).to(torch.float8_e4m3fn) for _ in range(2)]
    sc = [torch.ones((p, 2), device=cuda_dev) for _ in range(2)]
    ok = dict(k_scale=sc[0], v_scale=sc[1])
    plan.kv_append(k, k, *pages, table, **ok)

    def status(fn):
        with pytest.raises(msa.MsaError) as e:
            fn()
        return e.value.status
    assert status(lambda: plan.kv_append(k, k, pages[0], pages[0], table, **ok)) == 1
    assert status(lambda: plan.kv_append(k, k, *pages, table, k_scale=sc[0], v_scale=sc[0])) == 1
    assert status(lambda: plan.kv_append(k, k, *pages, table, rope=_rope(128), **ok)) == 1
    assert status(lambda: plan.append_bwd(table, dk_pages=torch.zeros((p, 2, 128, 64), device=cuda_dev))) == 2
    off = torch.zeros(4 * 128 + 4, device=cuda_dev).bfloat16()[4:].view(4, 2, 64)        # 8 bytes past a boundary
    assert status(lambda: plan.kv_append(off, k, *pages, table, **ok)) == 1
    for bad in (dict(k_scale=sc[0][:, 0], v_scale=sc[1]), dict(k_scale=sc[0], v_scale=sc[1][0])):
        with pytest.raises(ValueError):
            plan.kv_append(k, k, *pages, table, **bad)
    with pytest.raises(TypeError):
        plan.kv_append(k.float(), k, *pages, table, **ok)
    with pytest.raises(ValueError):
        plan.kv_append(k.transpose(1, 2).contiguous().transpose(1, 2), k, *pages, table, **ok)   # heads not dense
    pk = torch.zeros((4, 1, 32), device=cuda_dev).bfloat16()
    assert status(lambda: plan.pk_append(pk, table)) == 1
    assert status(lambda: plan.pk_append(pk, table, pk_pages_e4m3=torch.zeros(
        (p, 1, 128, 32), device=cuda_dev).to(torch.float8_e4m3fn))) == 1
    assert status(lambda: plan.pk_append(pk, table, pk_codes=torch.zeros(
        (p, 1, 128, 16), dtype=torch.uint8, device=cuda_dev))) == 1
    bfp = _msa().Plan([4], [4], 2, 2, 2, 64, 32, 1, p)
    assert status(lambda: bfp.append_bwd(table)) == 1
