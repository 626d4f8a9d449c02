"""The latent cache against its definitions in 64 bits: append, absorbed attention,
expansion, and the two forms of the attention against each other."""
import gc

import numpy as np
import pytest
import torch

from oracle import msa_oracle as O
from tests.tree_cases import attend, check, selection, tree_mask

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _collected():
    """Plans that a test's tracebacks hold go with it."""
    yield
    gc.collect()


def _msa():
    from block_sparse_long_proxy_gb300 import msa
    return msa


def _table(kv, extra, rng, dev):
    n = sum((k + 127) // 128 for k in kv)
    return torch.from_numpy(rng.permutation(n + extra)[:n].astype(np.int32)).to(dev), n + extra


def _holes(pages, table, kv, hidden=None):
    """NaN in pages that no table names and behind each last key, and at keys that are
    hidden ([sequence][key])."""
    keep, base = torch.zeros(pages.shape[:3], dtype=torch.bool, device=pages.device), 0
    for s, k in enumerate(kv):
        for j in range((k + 127) // 128):
            n = min(128, k - 128 * j)
            keep[int(table[base + j]), :, :n] = True
            for i in range(n):
                if hidden is not None and hidden[s][128 * j + i]:
                    keep[int(table[base + j]), :, i] = False
        base += (k + 127) // 128
    pages[~keep] = float("nan")


class Case:
    def __init__(self, dev, qo, kv, hq, hp, latent, rope, topk, tree, seed=0, grow=0.0, irregular=True):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.qo, self.kv, self.hq, self.hp, self.latent, self.rope, self.topk = qo, kv, hq, hp, latent, rope, topk
        self.table, self.p = _table(kv, 2, rng, dev)
        width = latent + rope
        self.mask = self.seen = None
        if tree:
            words, self.seen = tree_mask(qo, rng)
            self.mask = torch.from_numpy(words).to(dev)
        self.idx_h = selection(qo, kv, hp, topk, rng, irregular)
        self.q = torch.randn((sum(qo), hq, width), generator=gen, device=dev).to(torch.bfloat16)
        x = torch.randn((self.p, 1, 128, width), generator=gen, device=dev)
        if grow:
            f = torch.ones(self.p, device=dev)
            f[self.table.long()] = torch.cat([1 + grow * torch.arange((k + 127) // 128) for k in kv]).to(dev)
            x = x * f[:, None, None, None]
            self.idx_h.sort(-1)
        self.idx = torch.from_numpy(self.idx_h).to(dev)
        self.pages = x.to(torch.bfloat16)
        self.value = self.pages.double()
        hidden, r0 = [], 0
        for q, k in zip(qo, kv):
            h = np.zeros(k, bool)
            if tree:
                h[k - q:] = ~self.seen[r0:r0 + q, :q].any(0)
            hidden.append(h)
            r0 += q
        _holes(self.pages, self.table, kv, hidden)
        self.scale = 1.3 / np.sqrt(width)

    def plan(self):
        return _msa().Plan(self.qo, self.kv, self.hq, 1, self.hp, 128, 64, self.topk, self.p)

    def run(self, plan, **kw):
        return plan.latent_attn(self.q, self.pages, self.table, self.idx, self.rope, self.scale, tree_mask=self.mask, **kw)

    def ref(self):
        k = lambda e, h: self.value[int(self.table[e]), 0]  # noqa: E731
        return attend(self.q, k, lambda e, h: k(e, h)[:, :self.latent], self.qo, self.kv, self.idx_h,
                      float(np.float32(self.scale)), self.seen)

    def check(self, out, lse, ref):
        check(out, lse, ref, self.latent + 64, "latent", self.topk * 128)


SHAPES = {  # qo, kv, hq, hp, topk
    "one token": ([1], [1], 1, 1, 1),
    "decode": ([1] * 5, [128, 129, 300, 1, 1000], 16, 1, 5),
    "decode, 128 heads": ([1] * 3, [640, 1, 777], 128, 1, 4),
    "decode, 20 heads, two selections": ([1] * 4, [640, 5, 777, 256], 20, 2, 4),
    "few rows": ([5, 16, 2], [260, 16, 1000], 12, 4, 4),
    "long selection over a cluster": ([1], [128 * 40 + 5], 40, 1, 41),
}


@pytest.mark.parametrize("latent, rope", [(512, 64), (384, 48), (256, 32), (128, 16)])
@pytest.mark.parametrize("tree", [False, True], ids=["causal", "tree"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: s.replace(" ", "_"))
def test_absorbed(cuda_dev, shape, tree, latent, rope):
    qo, kv, hq, hp, topk = SHAPES[shape]
    c = Case(cuda_dev, qo, kv, hq, hp, latent, rope, topk, tree, seed=len(shape))
    plan = c.plan()
    out, lse = c.run(plan)
    plan.check_errors()
    c.check(out, lse, c.ref())


@pytest.mark.parametrize("qo, kv, hq, hp, topk", [([300, 128, 1, 130], [900, 128, 700, 131], 6, 2, 5), ([129], [257], 16, 1, 3)])
def test_causal_chunks(cuda_dev, qo, kv, hq, hp, topk):
    """Several tiles a sequence."""
    c = Case(cuda_dev, qo, kv, hq, hp, 256, 64, topk, False, seed=2)
    plan = c.plan()
    out, lse = c.run(plan)
    plan.check_errors()
    c.check(out, lse, c.ref())


@pytest.mark.parametrize("hq", [4, 24, 50])
def test_maxima_that_keep_moving(cuda_dev, hq):
    c = Case(cuda_dev, [1, 2], [3000, 2500], hq, 1, 512, 64, 24, False, seed=hq, grow=0.4, irregular=False)
    plan = c.plan()
    out, lse = c.run(plan)
    plan.check_errors()
    c.check(out, lse, c.ref())


def test_captures_and_streams(cuda_dev):
    """Two graphs and an eager call of one plan at once; the same bits from each."""
    c = Case(cuda_dev, [1] * 6, [900, 3000, 131, 2000, 77, 640], 32, 1, 512, 64, 8, False, seed=5)
    plan = c.plan()
    want = c.run(plan)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.run(plan))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
    with torch.cuda.stream(streams[2]):
        outs.append(c.run(plan))
    torch.cuda.synchronize()
    plan.check_errors()
    c.check(*want, c.ref())
    for out, lse in outs:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ------------------------------------------------------------------ append --

@pytest.mark.parametrize("latent, rope, rot, layout", [(512, 64, 64, "half"), (128, 16, 16, "interleaved"), (256, 48, 32, "half"),
                                                       (384, 64, None, None)])
@pytest.mark.parametrize("qo, kv", [([1] * 5, [1, 128, 129, 300, 257]), ([300, 5, 1], [1000, 5, 140]), ([20], [150])],
                         ids=["decode", "chunks", "across an edge"])
def test_append(cuda_dev, qo, kv, latent, rope, rot, layout):
    """Rows at strides, at positions of their own, into pages partly filled; all else
    keeps its bytes."""
    msa = _msa()
    rng = np.random.default_rng(3)
    gen = torch.Generator(device=cuda_dev).manual_seed(3)
    table, p = _table(kv, 2, rng, cuda_dev)
    rows = sum(qo)
    wide = torch.randn((rows, 24 + latent + rope), generator=gen, device=cuda_dev).to(torch.bfloat16)
    c, kr = wide[:, None, 8:8 + latent], wide[:, None, 16 + latent:16 + latent + rope]
    pages = torch.randn((p, 1, 128, latent + rope), generator=gen, device=cuda_dev).to(torch.bfloat16)
    before = pages.clone()
    plan = msa.Plan(qo, kv, 4, 1, 1, 128, 64, 1, p)
    r = msa.Rope(rot, layout) if rot else None
    pos = torch.from_numpy(rng.integers(0, 10 ** 6, rows).astype(np.int32)).to(cuda_dev)
    for positions in (pos, None):
        pages.copy_(before)
        plan.latent_append(c, kr, pages, table, rope=r, positions=positions)
        plan.check_errors()
        own = np.concatenate([np.arange(k - q, k) for q, k in zip(qo, kv)])
        x = kr.double().cpu().numpy()
        turned = O.rope(x, pos.cpu().numpy() if positions is not None else own, rot, layout) if rot else x
        want, base, i = before.clone(), 0, 0
        for q, k in zip(qo, kv):
            for key in range(k - q, k):
                page, slot = int(table[base + key // 128]), key % 128
                got = pages[page, 0, slot]
                assert torch.equal(got[:latent], c[i, 0])
                # an fp32 rotation (angles right to fp32: 2^-22 of |a| + |b|), rounded once to bf16
                t = turned[i, 0]
                far = np.abs(got[latent:].double().cpu().numpy() - t)
                size = np.abs(x[i]).max() * 2
                assert (far <= 2.0 ** -8 * np.abs(t) + (2.0 ** -21 * size if rot else 0.0)).all()
                want[page, 0, slot] = got
                i += 1
            base += (k + 127) // 128
        assert torch.equal(pages, want)


def test_append_bad_pages(cuda_dev):
    msa = _msa()
    plan = msa.Plan([3, 2], [100, 129], 4, 1, 1, 128, 64, 1, 4)
    pages = torch.zeros((4, 1, 128, 128 + 16), device=cuda_dev).bfloat16()
    c, kr = torch.ones((5, 1, 128), device=cuda_dev).bfloat16(), torch.ones((5, 1, 16), device=cuda_dev).bfloat16()
    table = torch.tensor([1, 4, -1], dtype=torch.int32, device=cuda_dev)
    plan.latent_append(c, kr, pages, table)
    with pytest.raises(msa.MsaError) as e:
        plan.check_errors()
    assert e.value.status == 6
    assert (pages[1, 0, 97:100] == 1).all() and pages.sum() == 3 * 144


# --------------------------------------------------------------- expansion --

@pytest.mark.parametrize("latent, rope, d", [(512, 64, 128), (128, 16, 64), (256, 32, 64), (384, 48, 128), (512, 16, 128)])
@pytest.mark.parametrize("kv, heads", [([1], 1), ([128, 129, 300], 5), ([700, 64], 16), ([130] * 90, 3)],
                         ids=["one key", "edges", "16 heads", "many pages"])
def test_expand(cuda_dev, kv, heads, latent, rope, d):
    msa = _msa()
    rng = np.random.default_rng(heads)
    gen = torch.Generator(device=cuda_dev).manual_seed(heads)
    rand = lambda *s: torch.randn(s, generator=gen, device=cuda_dev).to(torch.bfloat16)  # noqa: E731
    table, p = _table(kv, 2, rng, cuda_dev)
    c, w_k, w_v = rand(p, 1, 128, latent + rope), rand(heads, d - rope, latent), rand(heads, d, latent)
    whole = c.double()
    _holes(c, table, kv)
    k, v = rand(p, heads, 128, d), rand(p, heads, 128, d)
    old = k.clone(), v.clone()
    plan = msa.Plan([1] * len(kv), kv, heads, heads, heads, d, 64, 1, p)
    plan.latent_expand(c, w_k, w_v, table, k, v)
    plan.check_errors()
    there, base = torch.zeros((p, 128), dtype=torch.bool, device=cuda_dev), 0
    for n in kv:
        for j in range((n + 127) // 128):
            there[int(table[base + j]), :n - 128 * j] = True
        base += (n + 127) // 128
    for got, w, o, wide in ((k, w_k, old[0], d - rope), (v, w_v, old[1], d)):
        want = torch.einsum("ptc,hnc->phtn", whole[:, 0, :, :latent], w.double())
        size = torch.einsum("ptc,hnc->phtn", whole[:, 0, :, :latent].abs(), w.double().abs())
        # latent / 16 additions in fp32, then bf16
        tol = 2.0 ** -8 * want.abs() + latent / 16 * 2.0 ** -22 * size
        at = there[:, None, :, None]
        assert ((got[..., :wide].double() - want).abs() <= tol)[at.expand(-1, heads, -1, wide)].all()
        if wide < d:
            assert torch.equal(got[..., wide:][at.expand(-1, heads, -1, rope)], c[..., latent:].expand(-1, heads, -1, -1)[
                at.expand(-1, heads, -1, rope)])
        assert torch.equal(got[~there[:, None].expand(-1, heads, -1)], o[~there[:, None].expand(-1, heads, -1)])


@pytest.mark.parametrize("latent", [128, 384])
@pytest.mark.parametrize("rope, d", [(16, 64), (32, 64), (48, 64), (16, 128), (32, 128), (48, 128), (64, 128)])
def test_expand_of_every_width(cuda_dev, rope, d, latent):
    """Each split of a head's dims, whose products have 80 to 240 columns: several heads, so
    that both accumulators and all stages are used more than once."""
    test_expand(cuda_dev, [300, 5, 128], 7, latent, rope, d)


def test_expand_bad_pages(cuda_dev):
    msa = _msa()
    plan = msa.Plan([1], [300], 2, 2, 2, 64, 64, 1, 3)
    c, w = torch.ones((3, 1, 128, 144), device=cuda_dev).bfloat16(), torch.ones((2, 64, 128), device=cuda_dev).bfloat16()
    k, v = (torch.zeros((3, 2, 128, 64), device=cuda_dev).bfloat16() for _ in range(2))
    plan.latent_expand(c, w[:, :48].contiguous(), w, torch.tensor([2, 3, -7], dtype=torch.int32, device=cuda_dev), k, v)
    with pytest.raises(msa.MsaError) as e:
        plan.check_errors()
    assert e.value.status == 6
    assert (k[:2] == 0).all() and (v[:2] == 0).all() and (k[2, :, :, :48] == 128).all() and (v[2] == 128).all()


# ------------------------------------------------------- the two forms ----

@pytest.mark.parametrize("latent, rope, d", [(512, 64, 128), (256, 32, 64)])
def test_prefill_expanded_decode_absorbed(cuda_dev, latent, rope, d):
    """A prompt through the expanded form, then a decode step through the absorbed one
    over the same cache; each form against both, with the weights applied in 64 bits."""
    msa = _msa()
    gen = torch.Generator(device=cuda_dev).manual_seed(8)
    rand = lambda *s: torch.randn(s, generator=gen, device=cuda_dev).to(torch.bfloat16)  # noqa: E731
    heads, kv, topk, p, nope = 6, [300, 129], 3, 6, d - rope
    w_k, w_v = ((rand(heads, n, latent).float() / latent ** 0.5).to(torch.bfloat16) for n in (nope, d))
    pages = torch.zeros((p, 1, 128, latent + rope), device=cuda_dev).bfloat16()
    table = torch.tensor([4, 0, 2, 1, 5], dtype=torch.int32, device=cuda_dev)
    rope_h = msa.Rope(rope)
    rows = sum(kv)
    plan = msa.Plan(kv, kv, heads, heads, heads, d, 64, topk, p)
    c, kr = rand(rows, 1, latent), rand(rows, 1, rope)
    plan.latent_append(c, kr, pages, table, rope=rope_h)
    k_pages, v_pages = rand(p, heads, 128, d), rand(p, heads, 128, d)
    plan.latent_expand(pages, w_k, w_v, table, k_pages, v_pages)
    pos = torch.cat([torch.arange(n) for n in kv]).to(torch.int32).to(cuda_dev)
    q_nope, q_rope = rand(rows, heads, nope), rope_h.apply(rand(rows, heads, rope), pos)
    idx = torch.full((plan.n_tiles, heads, topk), -1, dtype=torch.int32, device=cuda_dev)
    for t, n in enumerate(plan.num_valid_pages.tolist()):
        idx[t, :, :n] = torch.arange(n)
    out, lse = plan.sparse_attn(torch.cat((q_nope, q_rope), -1), k_pages, v_pages, table, idx)
    plan.check_errors()
    # absorbed, over the same rows
    q_abs = torch.einsum("rhn,hnc->rhc", q_nope.double(), w_k.double()).to(torch.bfloat16)
    flat = msa.Plan(kv, kv, heads, 1, 1, 128, 64, topk, p)
    lat, lat_lse = flat.latent_attn(torch.cat((q_abs, q_rope), -1), pages, table, idx[:, :1].contiguous(), rope, d ** -0.5)
    flat.check_errors()
    got = torch.einsum("rhc,hnc->rhn", lat.double(), w_v.double())
    # K, V and q_abs are rounded to bf16 each (2^-8), as are weights and outputs of either form: a logit of size B
    # is off by 2^-8 B in each form, and an output by their sum and two roundings
    far = (got - out.double()).abs()
    assert far.mean() <= 0.02 * out.double().abs().mean() and far.max() <= 0.1 * out.double().abs().max()
    assert (lat_lse - lse).abs().max() <= 2 * 2.0 ** -8 * 4 * d ** 0.5
    # one more token
    one = msa.Plan([1, 1], [k + 1 for k in kv], heads, 1, 1, 128, 64, topk, p)
    one.latent_append(rand(2, 1, latent), rand(2, 1, rope), pages, table, rope=rope_h)
    q1 = rand(2, heads, latent + rope)
    i1 = torch.tensor([[[0, 1, 2]], [[0, 1, -1]]], dtype=torch.int32, device=cuda_dev)
    o1, l1 = one.latent_attn(q1, pages, table, i1, rope, 0.05)
    one.check_errors()
    k1 = lambda e, h: pages[int(table[e]), 0].double()  # noqa: E731
    ref = attend(q1, k1, lambda e, h: k1(e, h)[:, :latent], [1, 1], [k + 1 for k in kv], i1.cpu().numpy(), float(np.float32(0.05)))
    check(o1, l1, ref, latent + 64, "latent", topk * 128)


def test_refusals(cuda_dev):
    msa = _msa()
    c = Case(cuda_dev, [4], [200], 8, 1, 256, 32, 2, True)
    plan = c.plan()
    assert c.run(plan)[0].shape == (4, 8, 256)

    def status(fn):
        with pytest.raises(msa.MsaError) as e:
            fn()
        return e.value.status
    attn = lambda q=c.q, pages=c.pages, rope=32, scale=0.1, mask=c.mask: plan.latent_attn(  # noqa: E731
        q, pages, c.table, c.idx, rope, scale, tree_mask=mask)
    assert status(lambda: attn(rope=16)) == 2 and status(lambda: attn(rope=160)) == 2
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert status(lambda: attn(scale=s)) == 1
    long = msa.Plan([129], [200], 8, 1, 1, 128, 64, 2, c.p)
    z = lambda *s: torch.zeros(s, device=cuda_dev).bfloat16()  # noqa: E731
    assert status(lambda: long.latent_attn(z(129, 8, 288), c.pages, c.table, torch.zeros((2, 1, 2), dtype=torch.int32, device=cuda_dev),
                                           32, 0.1, tree_mask=torch.zeros((129, 4), dtype=torch.int32, device=cuda_dev))) == 2
    with pytest.raises(ValueError):
        attn(pages=c.pages[..., :280])
    with pytest.raises(TypeError):
        attn(q=c.q.float())
    rows = z(4, 1, 256), z(4, 1, 32)
    assert status(lambda: plan.latent_append(*rows, c.pages, c.table, rope=msa.Rope(48))) == 1
    assert status(lambda: plan.latent_append(rows[0][..., :200], rows[1], z(c.p, 1, 128, 232), c.table)) == 2
    assert status(lambda: plan.latent_append(z(4 * 256 + 4)[4:].view(4, 1, 256), rows[1], c.pages, c.table)) == 1
    k = z(c.p, 1, 128, 128)
    with pytest.raises(ValueError):
        plan.latent_expand(c.pages, z(1, 90, 256), z(1, 128, 256), c.table, k, k.clone())
    assert status(lambda: plan.latent_expand(c.pages, z(1, 96, 256), z(1, 128, 256), c.table, k, k)) == 1
    block = msa.Plan([1], [1], 2, 2, 2, 128, 64, 1, c.p, kv_dtype="e4m3_block")
    e4 = [torch.zeros((c.p, 2, 128, 128), device=cuda_dev).to(torch.float8_e4m3fn) for _ in range(2)]
    with pytest.raises((ValueError, TypeError, msa.MsaError)):
        block.latent_expand(c.pages, z(2, 96, 256), z(2, 128, 256), c.table, *e4)


def test_pools_beyond_4_gib(cuda_dev):
    """Append, attention and expansion on pages behind the 2^32nd byte, bit for bit as
    on small pools; other pages stay as they were."""
    msa = _msa()
    latent, rope, heads, d = 512, 64, 8, 128
    kv, n = [300, 129], 5
    far = 2 ** 32 // (128 * (latent + rope) * 2) + 7      # of the latents; K and V are larger
    got = []
    for pages in (n, far):
        gen = torch.Generator(device=cuda_dev).manual_seed(6)
        rand = lambda *s: torch.randn(s, generator=gen, device=cuda_dev).to(torch.bfloat16)  # noqa: E731
        pool = torch.zeros((pages, 1, 128, latent + rope), device=cuda_dev, dtype=torch.bfloat16)
        table = torch.tensor([4, 1, 0, 3, 2], dtype=torch.int32, device=cuda_dev) + (pages - n)
        plan = msa.Plan(kv, kv, heads, heads, heads, d, 64, 2, pages)
        plan.latent_append(rand(sum(kv), 1, latent), rand(sum(kv), 1, rope), pool, table, rope=msa.Rope(rope))
        one = msa.Plan([1, 1], kv, 16, 1, 1, d, 64, 3, pages)
        idx = torch.tensor([[[0, 1, 2]], [[0, 1, -1]]], dtype=torch.int32, device=cuda_dev)
        out, lse = one.latent_attn(rand(2, 16, latent + rope), pool, table, idx, rope, 0.05)
        k, v = (torch.zeros((pages, heads, 128, d), device=cuda_dev, dtype=torch.bfloat16) for _ in range(2))
        plan.latent_expand(pool, rand(heads, d - rope, latent), rand(heads, d, latent), table, k, v)
        plan.check_errors()
        one.check_errors()
        assert pages == n or not any(x[:n].any().item() for x in (pool, k, v))
        got.append((pool[-n:].clone(), out, lse, k[-n:].clone(), v[-n:].clone()))
        del pool, k, v
    assert all(a.any() and torch.equal(a, b) for a, b in zip(*got))


def test_nan_is_reported_under_checks(cuda_dev, monkeypatch):
    monkeypatch.setenv("MSA_CHECKS", "1")
    msa = _msa()
    c = Case(cuda_dev, [4], [200], 8, 1, 256, 32, 2, True, seed=2)
    plan = c.plan()
    c.run(plan)
    plan.check_errors()
    rows = torch.zeros((4, 1, 288), device=cuda_dev).bfloat16()
    for at in (10, 270):                                  # the latent; the key part
        rows.zero_()
        rows[3, 0, at] = float("nan")
        plan.latent_append(rows[..., :256], rows[..., 256:], c.pages, c.table)
        with pytest.raises(msa.MsaError) as e:
            plan.check_errors()
        assert e.value.status == 7
    rows.zero_()
    plan.latent_append(rows[..., :256], rows[..., 256:], c.pages, c.table)
    plan.check_errors()
    c.q[1, 2, 3] = float("nan")
    c.run(plan)
    with pytest.raises(msa.MsaError) as e:
        plan.check_errors()
    assert e.value.status == 7


def test_a_page_of_two_sequences(cuda_dev):
    """A shared prefix: expansion writes a page named twice with the same bits, call after
    call, and both sequences attend over it."""
    msa = _msa()
    gen = torch.Generator(device=cuda_dev).manual_seed(4)
    rand = lambda *s: torch.randn(s, generator=gen, device=cuda_dev).to(torch.bfloat16)  # noqa: E731
    kv, p, heads = [256 + 40, 256 + 7, 300], 8, 5
    table = torch.tensor([2, 5, 0, 2, 5, 1, 5, 2, 7], dtype=torch.int32, device=cuda_dev)
    c, w_k, w_v = rand(p, 1, 128, 576), rand(heads, 64, 512), rand(heads, 128, 512)
    plan = msa.Plan([1] * 3, kv, heads, heads, heads, 128, 64, 3, p)
    got = []
    for _ in range(3):
        k, v = torch.zeros((p, heads, 128, 128), device=cuda_dev).bfloat16(), torch.zeros((p, heads, 128, 128), device=cuda_dev).bfloat16()
        plan.latent_expand(c, w_k, w_v, table, k, v)
        got.append((k, v))
    plan.check_errors()
    assert all(torch.equal(a, b) for g in got[1:] for a, b in zip(got[0], g))
    single = torch.einsum("ptc,hnc->phtn", c[[2, 5], 0, :, :512].double(), w_v.double())
    assert (got[0][1][[2, 5]].double() - single).abs().max() <= 2.0 ** -8 * single.abs().max() + 1e-3


@pytest.mark.parametrize("hq", [3, 32, 50])
def test_first_places_empty(cuda_dev, hq):
    """Selections whose blocks all stand behind 32 empty places."""
    c = Case(cuda_dev, [1, 2], [128 * 11, 300], hq, 1, 256, 32, 70, False, seed=17, irregular=False)
    sel = np.full_like(c.idx_h, -1)
    sel[:, :, 37:49] = c.idx_h[:, :, :12]
    c.idx_h, c.idx = sel, torch.from_numpy(sel).to(cuda_dev)
    plan = c.plan()
    out, lse = c.run(plan)
    plan.check_errors()
    c.check(out, lse, c.ref())


def test_calls_that_feed_each_other(cuda_dev):
    """Append, attention and expansion in a chain without a pause, each one's output the next
    one's input: the bits of the chain that waits after every call."""
    m = _msa()
    rng, kv, latent, rope, d = np.random.default_rng(31), [700, 130, 2000], 256, 32, 64
    gen = torch.Generator(device=cuda_dev).manual_seed(31)
    table, p = _table(kv, 2, rng, cuda_dev)
    plan = m.Plan([1] * 3, kv, 8, 8, 8, d, 32, 4, p)
    idx = torch.from_numpy(selection([1] * 3, kv, 8, 4, rng)).to(cuda_dev)
    draw = lambda *shape: torch.randn(shape, generator=gen, device=cuda_dev).to(torch.bfloat16)  # noqa: E731
    pages0, q, key = draw(p, 1, 128, latent + rope), draw(3, 8, latent + rope), draw(3, 1, rope)
    w_k, w_v = draw(8, d - rope, latent), draw(8, d, latent)
    first = draw(3, 8, latent)
    turn = m.Rope(rope)
    ends = []
    for pause in (True, False):
        wait = torch.cuda.synchronize if pause else lambda: None
        pages, k, v = pages0.clone(), torch.zeros((p, 8, 128, d), dtype=torch.bfloat16, device=cuda_dev), None
        v, out = torch.zeros_like(k), first.clone()
        torch.cuda.synchronize()
        for _ in range(10):
            plan.latent_append(out[:, :1], key, pages, table, rope=turn)
            wait()
            out, _ = plan.latent_attn(q, pages, table, idx, rope, 0.06)
            wait()
            plan.latent_expand(pages, w_k, w_v, table, k, v)
            wait()
        plan.check_errors()
        ends.append((out, pages, k, v))
    for x, y in zip(*ends):
        assert torch.equal(x, y)


def test_other_tensors_after_accepted_ones(cuda_dev):
    """What was accepted of one call's tensors says nothing of others: each check again, in any order,
    and rows at another stride."""
    c = Case(cuda_dev, [2, 3], [300, 140], 4, 1, 256, 32, 3, True)
    plan = c.plan()
    want = c.run(plan)
    good = dict(q=c.q, latent_pages=c.pages, kv_indices=c.table, kv_block_indexes=c.idx, tree_mask=c.mask)
    for name, bad, error in [("q", c.q[:, :, :128], ValueError), ("q", c.q.float(), TypeError), ("q", c.q.cpu(), ValueError),
                             ("latent_pages", c.pages[:-1], ValueError), ("kv_indices", c.table.long(), TypeError),
                             ("kv_block_indexes", c.idx.transpose(0, 2), ValueError), ("tree_mask", c.mask[:1], ValueError),
                             ("q", c.q.transpose(0, 1).contiguous().transpose(0, 1), ValueError)]:
        with pytest.raises(error):
            plan.latent_attn(rope_dim=32, scale=c.scale, **dict(good, **{name: bad}))
        got = plan.latent_attn(rope_dim=32, scale=c.scale, **good)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ValueError):
        plan.latent_attn(rope_dim=300, scale=c.scale, **good)
    gen = torch.Generator(device=cuda_dev).manual_seed(3)
    new = torch.randn((5, 1, 3, 288), generator=gen, device=cuda_dev).to(torch.bfloat16)
    ends = []
    for dense in (True, False, True, False):
        pages, row = c.pages.clone(), new[:, :, 1].contiguous() if dense else new[:, :, 1]
        plan.latent_append(row[..., :256], row[..., 256:], pages, c.table)
        ends.append(pages.view(torch.int16))
    assert all(torch.equal(ends[0], x) for x in ends[1:]) and not torch.equal(ends[0], c.pages.view(torch.int16))
    plan.check_errors()
