"""msa_tree_attn against its definition in 64 bits: trees of every shape over the
three caches, what must not be read, clusters, captures, streams and bad pages."""
import gc

import numpy as np
import pytest
import torch

from tests.tree_cases import attend, chain_mask, check, selection, tree_mask

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _collected():
    """Plans that a test's tracebacks hold go with it."""
    yield
    gc.collect()


def _msa():
    from block_sparse_long_proxy_gb300 import msa
    return msa


class Case:
    """A batch of trees: caches with NaN wherever no row looks."""

    def __init__(self, dev, qo, kv, hq, hkv, hp, d, topk, kind, seed=0, grow=0.0, empty=0.1, irregular=True):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.qo, self.kv, self.hq, self.hkv, self.hp, self.d, self.topk, self.kind = qo, kv, hq, hkv, hp, d, topk, kind
        nb = [(k + 127) // 128 for k in kv]
        self.p = p = sum(nb) + 2
        table = rng.permutation(p)[:sum(nb)].astype(np.int32)
        self.table = torch.from_numpy(table).to(dev)
        words, self.seen = tree_mask(qo, rng, empty)
        self.mask = torch.from_numpy(words).to(dev)
        self.idx_h = selection(qo, kv, hp, topk, rng, irregular)
        self.idx = torch.from_numpy(self.idx_h).to(dev)
        self.q = torch.randn((sum(qo), hq, d), generator=gen, device=dev).to(torch.bfloat16)
        shape = (p, hkv, 128, d)
        self.pages, self.scales, self.values = [], [], []
        for which in range(2):
            x = torch.randn(shape, generator=gen, device=dev)
            if which == 0 and grow:  # later blocks' keys are larger: the running maximum keeps moving
                at = np.concatenate([np.arange(n) for n in nb])
                f = torch.ones(p, device=dev)
                f[self.table.long()] = torch.from_numpy(1 + grow * at).float().to(dev)
                x = x * f[:, None, None, None]
            if kind == "bf16":
                pages, scale = x.to(torch.bfloat16), None
                value = pages.double()
            else:
                pages = (x * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
                if kind == "e4m3":
                    scale = 0.012 * (1 + torch.rand(hkv, generator=gen, device=dev))
                    value = pages.double() * scale.double()[None, :, None, None]
                else:
                    scale = torch.exp2(torch.randint(-8, -4, (p, hkv), generator=gen, device=dev).float())
                    value = pages.double() * scale.double()[:, :, None, None]
            # NaN in pages that no table names, behind each last key, and at drafts that no row sees
            hole = torch.ones((p, 128), dtype=torch.bool, device=dev)
            base, r0 = 0, 0
            for q, k, n in zip(qo, kv, nb):
                hidden = ~self.seen[r0:r0 + q, :q].any(0)
                for j in range(n):
                    key = np.arange(128) + 128 * j
                    bad = key >= k
                    draft = (key >= k - q) & (key < k)
                    bad[draft] |= hidden[key[draft] - (k - q)]
                    hole[int(table[base + j])] = torch.from_numpy(bad).to(dev)
                base, r0 = base + n, r0 + q
            h = hole[:, None, :].expand(p, hkv, 128)
            if kind == "bf16":
                pages[h] = float("nan")
            else:
                pages.view(torch.uint8)[h] = 0x7F
            self.pages.append(pages)
            self.scales.append(scale)
            self.values.append(value)
        self.vmax = float(self.values[1].abs().max())

    def plan(self):
        return _msa().Plan(self.qo, self.kv, self.hq, self.hkv, self.hp, self.d, 64, self.topk, self.p, kv_dtype=self.kind)

    def run(self, plan, **kw):
        return plan.tree_attn(self.q, *self.pages, self.table, kw.pop("idx", self.idx), kw.pop("mask", self.mask),
                              k_scale=self.scales[0], v_scale=self.scales[1], **kw)

    def ref(self, idx=None, seen="tree"):
        m = self.hp // self.hkv
        of = lambda x: lambda e, h: x[int(self.table[e]), h // m]  # noqa: E731
        return attend(self.q, of(self.values[0]), of(self.values[1]), self.qo, self.kv,
                      self.idx_h if idx is None else idx, self.d ** -0.5, self.seen if seen == "tree" else seen)

    def check(self, out, lse, ref):
        n = self.topk * 128
        check(out, lse, ref, self.d, self.kind, n, 0.0 if self.kind == "bf16" else 2.0 ** -25 * n * self.vmax * 16)


# 16 in `room` above: the largest weight belongs to a page whose value scale may be 8 times smaller than
# the largest one's, and to a code of half of 448


SHAPES = {  # qo, kv, hq, hkv, hp, topk
    "one draft, nothing before": ([1], [1], 8, 8, 8, 1),
    "one row each": ([1] * 5, [128, 129, 300, 1, 1000], 8, 2, 2, 5),
    "from the page's edge": ([16, 16, 17, 3], [128 + 16, 127 + 16, 255 + 17, 130], 16, 2, 2, 3),
    "across an edge, three heads": ([61, 2, 40], [700, 2, 1290], 12, 4, 4, 4),
    "two selections a KV head": ([7, 30], [900, 333], 16, 2, 4, 6),
    "nothing before": ([128, 128, 33, 1], [128, 200, 33, 2], 4, 4, 4, 2),
    "widest trees, one head": ([128, 100], [128 * 5 + 1, 777], 2, 2, 2, 9),
    "widest trees, 16 heads": ([128], [1500], 32, 2, 2, 12),
    "a long selection over a cluster": ([9], [128 * 70 + 5], 8, 1, 1, 70),
    "five heads": ([13] * 3, [600, 13, 140], 20, 4, 4, 3),
    "sequences without rows": ([0, 5, 0, 2], [10, 300, 400, 129], 6, 2, 2, 2),
}


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3_block"])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: s.replace(" ", "_"))
def test_trees(cuda_dev, shape, d, kind):
    qo, kv, hq, hkv, hp, topk = SHAPES[shape]
    c = Case(cuda_dev, qo, kv, hq, hkv, hp, d, topk, kind, seed=len(shape))
    plan = c.plan()
    out, lse = c.run(plan)
    plan.check_errors()
    c.check(out, lse, c.ref())


WIDE = {  # batches whose (row, head) pairs fill the rows of the products (test_tree_latent_host.py)
    "ragged": ([64, 100, 37, 128, 5, 128, 90, 128, 128, 65, 128, 33, 128, 128, 128, 128],
               [700, 100, 300, 1000, 900, 128, 219, 1281, 640, 65, 777, 1290, 128 * 9 + 3, 500, 256, 131], 32, 4, 4, 5),
    "odd heads, two selections": ([128] * 14, [300 + 97 * i for i in range(14)], 48, 4, 8, 7),
}


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3_block"])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("shape", WIDE, ids=lambda s: s.replace(" ", "_"))
def test_wide_trees(cuda_dev, shape, d, kind):
    qo, kv, hq, hkv, hp, topk = WIDE[shape]
    for grow in (0.0, 0.4):
        c = Case(cuda_dev, qo, kv, hq, hkv, hp, d, topk, kind, seed=len(shape), grow=grow)
        if grow:
            c.idx_h.sort(-1)
            c.idx = torch.from_numpy(c.idx_h).to(cuda_dev)
        plan = c.plan()
        out, lse = c.run(plan)
        plan.check_errors()
        c.check(out, lse, c.ref())


def test_wide_trees_bad_pages(cuda_dev):
    """As test_bad_pages_are_skipped_and_reported, over batches of wide trees."""
    qo, kv, hq, hkv, hp, topk = WIDE["ragged"]
    c = Case(cuda_dev, qo, kv, hq, hkv, hp, 128, topk, "bf16", seed=2, irregular=False)
    table = c.table.cpu().numpy().copy()
    bad = np.random.default_rng(5).random(table.size) < 0.2
    ids = np.where(bad, -3, table).astype(np.int32)
    named, base = c.idx_h.copy(), np.concatenate([[0], np.cumsum([(k + 127) // 128 for k in kv])])
    for t in range(len(qo)):
        sel = named[t]
        sel[(sel >= 0) & bad[base[t] + np.maximum(sel, 0)]] = -1
    plan, good = c.plan(), c.table
    c.table = torch.from_numpy(ids).to(cuda_dev)
    out, lse = c.run(plan)
    with pytest.raises(_msa().MsaError) as e:
        plan.check_errors()
    assert e.value.status == 6
    c.table = good
    c.check(out, lse, c.ref(idx=named))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3_block"])
@pytest.mark.parametrize("rows", [1, 3, 8, 40])
def test_maxima_that_keep_moving(cuda_dev, rows, kind):
    """Keys that grow from block to block: sums and outputs are rescaled at many."""
    c = Case(cuda_dev, [rows] * 2, [3000, 2500], 8, 2, 2, 128, 24, kind, seed=rows, grow=0.4, irregular=False)
    c.idx_h.sort(-1)
    c.idx = torch.from_numpy(c.idx_h).to(cuda_dev)
    plan = c.plan()
    out, lse = c.run(plan)
    plan.check_errors()
    c.check(out, lse, c.ref())


def test_chain_is_the_causal_attention(cuda_dev):
    """A tree that is a chain has the rows of msa_sparse_attn."""
    c = Case(cuda_dev, [30, 5], [900, 260], 16, 4, 4, 128, 4, "bf16", seed=3, empty=0.0)
    c.pages = [torch.nan_to_num(p) for p in c.pages]
    mask = torch.from_numpy(chain_mask(c.qo)).to(cuda_dev)
    plan = c.plan()
    out, lse = c.run(plan, mask=mask)
    want, want_lse = plan.sparse_attn(c.q, *c.pages, c.table, c.idx)
    plan.check_errors()
    c.check(out, lse, c.ref(seen=None))
    fin = torch.isfinite(want_lse)
    assert torch.equal(torch.isfinite(lse), fin) and (lse - want_lse)[fin].abs().max() <= 1e-4
    # both sides round weights and outputs to bf16
    assert (out.float() - want.float()).abs().max() <= 2 * 2.0 ** -8 * 2 * c.vmax


def test_outputs_given_streams_and_repeats(cuda_dev):
    """Given outputs, no lse, another stream, two calls of a plan at once, and the same
    bits every time."""
    c = Case(cuda_dev, [16] * 4, [900, 3000, 131, 2000], 16, 2, 2, 128, 16, "e4m3_block", seed=9)
    plan = c.plan()
    out, lse = c.run(plan)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    others = []
    torch.cuda.synchronize()
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            others.append(c.run(plan))
    c.run(plan, out=o2, lse=l2, stream=streams[0])
    torch.cuda.synchronize()
    plan.check_errors()
    c.check(out, lse, c.ref())
    for a, b in others + [(o2, l2)]:
        assert torch.equal(a, out) and torch.equal(b, lse)
    o3, none = c.run(plan, want_lse=False)
    assert none is None and torch.equal(o3, out)


def test_captured_and_replayed(cuda_dev):
    """Two graphs of one plan, replayed at once, on inputs that change in place."""
    c = Case(cuda_dev, [8] * 3, [700, 1500, 260], 16, 2, 2, 128, 8, "bf16", seed=4)
    plan = c.plan()
    c.run(plan)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.run(plan))
        graphs.append(g)
    gen = torch.Generator(device=cuda_dev).manual_seed(77)
    c.q.copy_(torch.randn(c.q.shape, generator=gen, device=cuda_dev))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    plan.check_errors()
    ref = c.ref()
    for out, lse in outs:
        c.check(out, lse, ref)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3_block"])
def test_bad_pages_are_skipped_and_reported(cuda_dev, kind):
    """Blocks on pages outside the pool, and blocks behind a tile's last, count as not
    selected."""
    c = Case(cuda_dev, [16, 4], [128 * 9 + 7, 650], 16, 2, 2, 128, 8, kind, seed=6, irregular=False)
    rng = np.random.default_rng(8)
    table = c.table.cpu().numpy().copy()
    bad = rng.random(table.size) < 0.3
    bad[0] = True
    ids = np.where(bad, rng.choice([-1, -2 ** 31, c.p, 2 ** 31 - 1, 2 ** 24], table.size), table).astype(np.int32)
    base = np.array([0, 10])
    named = c.idx_h.copy()
    named[(named >= 0) & bad[base[:, None, None] + np.maximum(named, 0)]] = -1
    sel = c.idx_h.copy()
    sel[1, 0, np.argmax(sel[1, 0] < 0)] = 6              # the sequence has blocks 0..5
    plan = c.plan()
    good = c.table
    c.table = torch.from_numpy(ids).to(cuda_dev)
    out, lse = c.run(plan, idx=torch.from_numpy(sel).to(cuda_dev))
    with pytest.raises(_msa().MsaError) as e:
        plan.check_errors()
    assert e.value.status == 6
    c.table = good
    c.check(out, lse, c.ref(idx=named))


def test_draft_step(cuda_dev):
    """A step as a server takes it: drafts appended at their places in the text,
    blocks scored and selected, the tree attended, and the accepted path appended
    again; the cache is then that of the tokens taken one by one."""
    msa = _msa()
    gen = torch.Generator(device=cuda_dev).manual_seed(1)
    ctx, d, hkv, hq, topk = [300, 1000], 128, 2, 16, 4
    parent = [[-1, 0, 0, 1, 2, 2, 4], [-1, -1, 0, 1, 3]]
    depth = [[0, 1, 1, 2, 2, 2, 3], [0, 0, 1, 1, 2]]
    taken = [[0, 2, 4, 6], [1, 3]]
    qo = [len(p) for p in parent]
    nb = [(c + 128 + 127) // 128 for c in ctx]
    p, rows = sum(nb), sum(qo)
    rand = lambda *s: torch.randn(s, generator=gen, device=cuda_dev).to(torch.bfloat16)  # noqa: E731
    tables = lambda kv: torch.cat([torch.arange(sum(nb[:s]), sum(nb[:s]) + (kv[s] + 127) // 128) for s in range(2)]).to(  # noqa: E731
        torch.int32).to(cuda_dev)
    k_pages, v_pages, pk_pages = rand(p, hkv, 128, d), rand(p, hkv, 128, d), rand(p, 1, 128, 64)
    k, v, pk = rand(rows, hkv, d), rand(rows, hkv, d), rand(rows, 1, 64)
    q, pq = rand(rows, hq, d), rand(rows, hkv, 64)
    rope, prope = msa.Rope(d), msa.Rope(64)
    seen = np.zeros((rows, 128), bool)
    r0 = 0
    for par in parent:
        for i, a in enumerate(par):
            if a >= 0:
                seen[r0 + i] = seen[r0 + a]
            seen[r0 + i, i] = True
        r0 += len(par)
    words = (seen.reshape(-1, 4, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)
    pos = torch.tensor([c + x for c, dd in zip(ctx, depth) for x in dd], dtype=torch.int32, device=cuda_dev)

    kv = [c + n for c, n in zip(ctx, qo)]
    plan = msa.Plan(qo, kv, hq, hkv, hkv, d, 64, topk, p)
    table = tables(kv)
    old_k, old_v = k_pages.clone(), v_pages.clone()
    plan.kv_append(k, v, k_pages, v_pages, table, rope=rope, positions=pos)
    plan.pk_append(pk, table, pk_pages=pk_pages, rope=prope, positions=pos)
    qr, pqr = rope.apply(q, pos), prope.apply(pq, pos)
    score = plan.proxy_maxscore(pqr, pk_pages, table)
    idx = msa.topk_select(score, topk, plan.num_valid_pages)
    out, lse = plan.tree_attn(qr, k_pages, v_pages, table, idx, torch.from_numpy(words).to(cuda_dev))
    plan.check_errors()
    of = lambda x: lambda e, h: x[int(table[e]), h].double()  # noqa: E731
    ref = attend(qr, of(k_pages), of(v_pages), qo, kv, idx.cpu().numpy(), d ** -0.5, seen)
    check(out, lse, ref, d, "bf16", topk * 128)

    # a draft's row is that of its path alone, over the same blocks
    kt, vt = old_k.clone(), old_v.clone()
    n = [len(t) for t in taken]
    at = torch.tensor([sum(qo[:s]) + i for s in range(2) for i in taken[s]], device=cuda_dev)
    kv1 = [c + m for c, m in zip(ctx, n)]
    step = msa.Plan(n, kv1, hq, hkv, hkv, d, 64, topk, p)
    step.kv_append(k[at], v[at], kt, vt, tables(kv1), rope=rope)
    same, _ = step.sparse_attn(qr[at], kt, vt, tables(kv1), idx)
    o, _, a, _ = ref
    assert ((same.double() - o[at]).abs() <= 2.0 ** -7 * a[at] + 2.0 ** -8 * o[at].abs()).all()
    # the accepted rows behind the context, as their tokens one by one would have left them
    accept = msa.Plan(n, kv1, hq, hkv, hkv, d, 64, topk, p)
    accept.kv_append(k[at], v[at], k_pages, v_pages, tables(kv1), rope=rope)
    for s in range(2):
        for i in range(ctx[s], kv1[s]):
            page, slot = sum(nb[:s]) + i // 128, i % 128
            assert torch.equal(k_pages[page, :, slot], kt[page, :, slot]) and torch.equal(v_pages[page, :, slot], vt[page, :, slot])


@pytest.mark.parametrize("form", ["tree", "latent"])
def test_drafts_across_a_page_edge(cuda_dev, form):
    """Drafts in two blocks, the first of which scores least of all: selected as it is, they
    lose the drafts there, and those their own keys; with its score set to inf, as the header
    says, every row sees its ancestors and itself, and each of them counts."""
    msa = _msa()
    gen = torch.Generator(device=cuda_dev).manual_seed(12)
    d, hkv, hq, topk, latent, turned = 64, 1, 8, 3, 128, 32
    parent = [-1, 0, 0, 1, 2, 4, 5, 3]
    qo, kv = [8, 8, 8], [128 * 6 + 3, 128 * 6, 128 * 6 + 8]     # five drafts before an edge; up to one; from one on
    n = sum(qo)
    seen = np.zeros((8, 128), bool)
    for i, a in enumerate(parent):
        if a >= 0:
            seen[i] = seen[a]
        seen[i, i] = True
    seen = np.concatenate([seen] * 3)
    words = torch.from_numpy((seen.reshape(-1, 4, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(
        np.uint32).view(np.int32)).to(cuda_dev)
    rand = lambda *s: torch.randn(s, generator=gen, device=cuda_dev).to(torch.bfloat16)  # noqa: E731
    nb = [(k + 127) // 128 for k in kv]
    table = torch.randperm(sum(nb), generator=gen, device=cuda_dev).to(torch.int32)
    plan = msa.Plan(qo, kv, hq, hkv, hkv, d, 64, topk, sum(nb))
    pos0 = [k - q for q, k in zip(qo, kv)]
    first = [p // 128 for p in pos0]
    score = torch.rand((3, 1, plan.max_blocks), generator=gen, device=cuda_dev)
    score[torch.arange(3), 0, first] = -1.0
    if form == "tree":
        q, k, v = rand(n, hq, d), rand(sum(nb), hkv, 128, d), rand(sum(nb), hkv, 128, d)
        scale, width, wide = d ** -0.5, d, d
        run = lambda idx: plan.tree_attn(q, k, v, table, idx, words)  # noqa: E731
        k_of, v_of = (lambda x: lambda e, h: x[int(table[e]), h].double())(k), (lambda x: lambda e, h: x[int(table[e]), h].double())(v)
    else:
        q, pages = rand(n, hq, latent + turned), rand(sum(nb), 1, 128, latent + turned)
        scale, width, wide = 0.125, latent + 64, latent
        run = lambda idx: plan.latent_attn(q, pages, table, idx, turned, scale, tree_mask=words)  # noqa: E731
        k_of = lambda e, h: pages[int(table[e]), 0].double()  # noqa: E731
        v_of = lambda e, h: k_of(e, h)[:, :latent]  # noqa: E731
    for keep in (False, True):
        if keep:
            score[torch.arange(3), 0, first] = float("inf")
        idx = msa.topk_select(score, topk, plan.num_valid_pages)
        got = idx.cpu().numpy()
        for t in range(3):
            assert nb[t] - 1 in got[t, 0] and (first[t] in got[t, 0]) == (keep or first[t] == nb[t] - 1)
        out, lse = run(idx)
        plan.check_errors()
        ref = attend(q, k_of, v_of, qo, kv, got, scale, seen)
        check(out, lse, ref, width, "bf16" if form == "tree" else "latent", topk * 128)
        # each draft's own key takes part: its value, times the weight, is what leaving it out would move
        alone = seen.copy()
        alone[np.arange(n), np.tile(np.arange(8), 3)] = False
        moved = (attend(q, k_of, v_of, qo, kv, got, scale, alone)[0] - ref[0]).abs().amax((1, 2)).cpu().numpy()
        lost = np.concatenate([[p + i < 128 * (b - 1) for i in range(8)] for p, b in zip(pos0, nb)])
        assert lost.sum() == 5 and ((moved == 0) == (lost & (not keep))).all()


def test_refusals(cuda_dev):
    msa = _msa()
    c = Case(cuda_dev, [4], [200], 8, 2, 2, 128, 2, "bf16")
    plan = c.plan()

    def status(fn):
        with pytest.raises(msa.MsaError) as e:
            fn()
        return e.value.status
    long = Case(cuda_dev, [100], [200], 8, 2, 2, 128, 2, "bf16")
    wide = msa.Plan([129], [200], 8, 2, 2, 128, 64, 2, long.p)
    q = torch.zeros((129, 8, 128), device=cuda_dev).bfloat16()
    mask = torch.zeros((129, 4), dtype=torch.int32, device=cuda_dev)
    idx = torch.zeros((2, 2, 2), dtype=torch.int32, device=cuda_dev)
    assert status(lambda: wide.tree_attn(q, *long.pages, long.table, idx, mask)) == 2
    assert status(lambda: plan.tree_attn(c.q, *c.pages, c.table, c.idx, c.mask, k_scale=torch.ones(2, device=cuda_dev),
                                         v_scale=torch.ones(2, device=cuda_dev))) == 1
    with pytest.raises(TypeError):
        plan.tree_attn(c.q, *c.pages, c.table, c.idx, c.mask.long())
    for bad in (c.mask[:, :2].contiguous(), c.mask[:2].contiguous(), c.mask.repeat(1, 2)[:, :4]):
        with pytest.raises(ValueError):
            plan.tree_attn(c.q, *c.pages, c.table, c.idx, bad)
    off = torch.zeros(c.q.numel() + 4, device=cuda_dev).bfloat16()[4:].view(c.q.shape)
    assert status(lambda: plan.tree_attn(off, *c.pages, c.table, c.idx, c.mask)) == 1


@pytest.mark.parametrize("kind, d, rows", [("bf16", 128, 5), ("e4m3", 128, 5), ("e4m3_block", 64, 5), ("bf16", 128, 100),
                                           ("e4m3_block", 128, 100)])
def test_pools_beyond_4_gib(cuda_dev, kind, d, rows):
    """Pages behind the 2^32nd byte, bit for bit as out of a small pool."""
    msa = _msa()
    hkv, hq, size = 8, 64, 2 if kind == "bf16" else 1
    far = 2 ** 32 // (hkv * 128 * d * size) + 5
    batch = 2 if rows == 5 else 16                        # columns; rows
    kv = [rows + 400 + i for i in range(batch)]
    gen = torch.Generator(device=cuda_dev).manual_seed(3)
    nb = sum((k + 127) // 128 for k in kv)
    small = [torch.randint(0, 120, (nb, hkv, 128, d * size), generator=gen, device=cuda_dev, dtype=torch.uint8) for _ in "kv"]
    if kind == "bf16":
        small = [torch.randn((nb, hkv, 128, d), generator=gen, device=cuda_dev).to(torch.bfloat16) for _ in "kv"]
    q = torch.randn((rows * batch, hq, d), generator=gen, device=cuda_dev).to(torch.bfloat16)
    words, _ = tree_mask([rows] * batch, np.random.default_rng(1))
    idx = torch.from_numpy(selection([rows] * batch, kv, hkv, 3, np.random.default_rng(2))).to(cuda_dev)
    got = []
    for pages in (nb, far):
        pools = []
        for x in small:
            pool = torch.zeros((pages, *x.shape[1:]), dtype=x.dtype, device=cuda_dev)
            pool[-nb:] = x
            pools.append(pool if kind == "bf16" else pool.view(torch.float8_e4m3fn))
        scale = None if kind == "bf16" else torch.full((hkv,) if kind == "e4m3" else (pages, hkv), 0.01, device=cuda_dev)
        plan = msa.Plan([rows] * batch, kv, hq, hkv, hkv, d, 64, 3, pages, kv_dtype=kind)
        table = torch.arange(pages - nb, pages, dtype=torch.int32, device=cuda_dev)
        got.append(plan.tree_attn(q, *pools, table, idx, torch.from_numpy(words).to(cuda_dev), k_scale=scale, v_scale=scale))
        plan.check_errors()
        del pools, pool
    assert got[0][0].any() and all(torch.equal(a, b) for a, b in zip(*got))


def test_nan_is_reported_under_checks(cuda_dev, monkeypatch):
    """MSA_CHECKS: a NaN among the queries is reported; one where no row looks is not."""
    monkeypatch.setenv("MSA_CHECKS", "1")
    c = Case(cuda_dev, [8, 3], [300, 40], 16, 2, 2, 128, 3, "bf16", seed=1)
    plan = c.plan()
    c.run(plan)
    plan.check_errors()
    c.q[2, 1, 5] = float("nan")
    c.run(plan)
    with pytest.raises(_msa().MsaError) as e:
        plan.check_errors()
    assert e.value.status == 7


def test_mask_of_any_alignment(cuda_dev):
    """tree_mask needs 4-byte alignment only, for rows as for columns."""
    for qo, kv, hq, hkv, hp, topk in (SHAPES["across an edge, three heads"], WIDE["ragged"]):
        c = Case(cuda_dev, qo, kv, hq, hkv, hp, 128, topk, "bf16", seed=8)
        plan = c.plan()
        want = c.run(plan)
        buf = torch.zeros(c.mask.numel() + 1, dtype=torch.int32, device=cuda_dev)
        off = buf[1:].view(c.mask.shape)
        off.copy_(c.mask)
        got = c.run(plan, mask=off)
        plan.check_errors()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_host_threads(cuda_dev):
    """Calls of two plans from two host threads at once, first calls among them."""
    import threading
    cases = [Case(cuda_dev, [7, 30], [900, 333], 16, 2, 4, 128, 6, "bf16", seed=4),
             Case(cuda_dev, *[[x for x in v] if isinstance(v, list) else v for v in WIDE["ragged"][:5]], 128, 5, "e4m3_block", seed=5)]
    out, errors = [None, None], []

    def work(i):
        try:
            torch.cuda.set_device(cuda_dev)
            with torch.cuda.stream(torch.cuda.Stream()):
                plan = cases[i].plan()
                for _ in range(20):
                    out[i] = cases[i].run(plan)
                torch.cuda.current_stream().synchronize()
                plan.check_errors()
        except Exception as e:                           # noqa: BLE001
            errors.append(e)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for c, (o, l) in zip(cases, out):
        c.check(o, l, c.ref())


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3_block"])
@pytest.mark.parametrize("rows", [1, 5, 14, 100])
def test_first_places_empty(cuda_dev, rows, kind):
    """Selections whose blocks all stand behind 32 empty places."""
    c = Case(cuda_dev, [rows] * 2, [rows + 128 * 11, rows + 300], 8, 1, 1, 128, 70, kind, seed=17, irregular=False)
    sel = np.full_like(c.idx_h, -1)
    sel[:, :, 37:49] = c.idx_h[:, :, :12]
    assert (sel[:, :, :37] == -1).all() and (sel[1] >= 0).sum() >= 3
    plan = c.plan()
    out, lse = c.run(plan, idx=torch.from_numpy(sel).to(cuda_dev))
    plan.check_errors()
    c.check(out, lse, c.ref(idx=sel))


@pytest.mark.parametrize("kind", ["bf16", "e4m3_block"])
@pytest.mark.parametrize("rows", [2, 40])
def test_calls_that_feed_each_other(cuda_dev, rows, kind):
    """A chain of calls without a pause, each one's output the next one's queries: the bits of
    the chain that waits after every call."""
    c = Case(cuda_dev, [rows] * 3, [900, 3000, 650], 16, 2, 2, 128, 6, kind, seed=21)
    plan = c.plan()
    ends = []
    for pause in (True, False):
        a, b = c.q.clone(), torch.zeros_like(c.q)
        torch.cuda.synchronize()
        for _ in range(20):
            plan.tree_attn(a, *c.pages, c.table, c.idx, c.mask, k_scale=c.scales[0], v_scale=c.scales[1], out=b,
                           want_lse=False)
            a, b = b, a
            if pause:
                torch.cuda.synchronize()
        plan.check_errors()
        ends.append(a.clone())
    assert torch.equal(*ends)
