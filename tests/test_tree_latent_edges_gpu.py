"""Tree and latent calls at the ends of what the header allows: the longest selections, rows
that are not finite, queries beyond f16, scales beyond their range, plans of other caches,
sequences without rows."""
import gc

import numpy as np
import pytest
import torch

from tests import test_latent_gpu, test_tree_attn_gpu
from tests.test_latent_gpu import _holes, _table

pytestmark = pytest.mark.gpu
TREES = {"columns": ([9, 5, 2], [700, 300, 130], 12, 2, 2, 4), "wide": test_tree_attn_gpu.WIDE["ragged"]}


@pytest.fixture(autouse=True)
def _collected():
    """Plans that a test's tracebacks hold go with it."""
    yield
    gc.collect()


def _msa():
    from block_sparse_long_proxy_gb300 import msa
    return msa


def _tree(dev, which, kind, d=128, seed=4):
    qo, kv, hq, hkv, hp, topk = TREES[which]
    return test_tree_attn_gpu.Case(dev, qo, kv, hq, hkv, hp, d, topk, kind, seed=seed)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3_block"])
@pytest.mark.parametrize("rows, hq", [(1, 4), (6, 12), (40, 4)])
def test_longest_selections_of_trees(cuda_dev, rows, hq, kind):
    """1024 blocks of 1026."""
    c = test_tree_attn_gpu.Case(cuda_dev, [rows], [128 * 1025 + 70], hq, 1, 1, 64, 1024, kind, seed=rows)
    plan = c.plan()
    out, lse = c.run(plan)
    plan.check_errors()
    c.check(out, lse, c.ref())


@pytest.mark.parametrize("latent, rows, hq", [(512, 1, 8), (128, 3, 16), (256, 5, 20)])
def test_longest_selections_of_latents(cuda_dev, latent, rows, hq):
    c = test_latent_gpu.Case(cuda_dev, [rows], [128 * 1025 + 70], hq, 1, latent, 64, 1024, False, seed=rows)
    plan = c.plan()
    out, lse = c.run(plan)
    plan.check_errors()
    c.check(out, lse, c.ref())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38], ids=str)
@pytest.mark.parametrize("which, kind", [("columns", "bf16"), ("columns", "e4m3_block"), ("wide", "bf16"), ("wide", "e4m3")])
def test_rows_of_trees_do_not_touch_each_other(cuda_dev, which, kind, bad):
    """A query that is not finite, or whose logits overflow, changes no other row and head."""
    c = _tree(cuda_dev, which, kind)
    plan = c.plan()
    want = c.run(plan)
    rng = np.random.default_rng(1)
    hit = torch.from_numpy(rng.random((sum(c.qo), c.hq)) < 0.2).to(cuda_dev)
    c.q[hit] = bad
    got = c.run(plan)
    plan.check_errors()
    assert hit.any() and all(torch.equal(a[~hit], b[~hit]) for a, b in zip(got, want))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38], ids=str)
@pytest.mark.parametrize("hq", [12, 32])
def test_rows_of_latents_do_not_touch_each_other(cuda_dev, hq, bad):
    c = test_latent_gpu.Case(cuda_dev, [9, 150, 2], [700, 300, 130], hq, 1, 256, 32, 4, False, seed=4)
    plan = c.plan()
    want = c.run(plan)
    rng = np.random.default_rng(1)
    hit = torch.from_numpy(rng.random((161, hq)) < 0.2).to(cuda_dev)
    c.q[hit] = bad
    got = c.run(plan)
    plan.check_errors()
    assert all(torch.equal(a[~hit], b[~hit]) for a, b in zip(got, want))


@pytest.mark.parametrize("kind, d", [("e4m3", 128), ("e4m3", 64), ("e4m3_block", 128)])
@pytest.mark.parametrize("which", ["columns", "wide"])
def test_queries_beyond_f16_saturate(cuda_dev, which, kind, d):
    """Whatever lies beyond 65504 counts as 65504."""
    c = _tree(cuda_dev, which, kind, d)
    c.scales[0] *= 2.0 ** -14
    plan = c.plan()
    got = []
    for big in (65504.0, 1e5, 3e38, float("inf")):
        c.q[..., 5], c.q[..., 40] = big, -big
        if big == 65504.0:                                # not a bf16: the next below and the next above
            c.q[..., 5], c.q[..., 40] = 65536.0, -65536.0
        got.append(c.run(plan))
    plan.check_errors()
    assert torch.isfinite(got[0][0]).all() and not torch.isnan(got[0][1]).any()
    assert all(torch.equal(x, y) for g in got[1:] for x, y in zip(g, got[0]))


@pytest.mark.parametrize("kind", ["e4m3", "e4m3_block"])
@pytest.mark.parametrize("which", ["columns", "wide"])
def test_scales_beyond_their_range(cuda_dev, which, kind):
    """Scales count as lying in [2^-40, 2^40], NaN and zero as the lower end."""
    c = _tree(cuda_dev, which, kind)
    plan = c.plan()
    rng = np.random.default_rng(2)
    odd = torch.tensor([0.0, -1.0, 2.0 ** -50, float("nan"), 1e-45, 2.0 ** -40], device=cuda_dev)
    for s in c.scales:
        pick = torch.from_numpy(rng.integers(0, len(odd), tuple(s.shape))).to(cuda_dev)
        some = torch.from_numpy(rng.random(tuple(s.shape)) < 0.4).to(cuda_dev)
        s[some] = odd[pick][some]
    got = c.run(plan)
    c.scales = [torch.where(s >= 2.0 ** -40, s, 2.0 ** -40) for s in c.scales]
    want = c.run(plan)
    plan.check_errors()
    assert torch.isfinite(got[0]).all() and all(torch.equal(a, b) for a, b in zip(got, want))


def test_latents_by_plans_of_other_caches(cuda_dev):
    """The plan's num_kv_heads, head_dim and kv_dtype are not read."""
    c = test_latent_gpu.Case(cuda_dev, [3, 140], [500, 260], 16, 2, 256, 32, 3, False, seed=6)
    want = c.run(c.plan())
    gen = torch.Generator(device=cuda_dev).manual_seed(6)
    row = torch.randn((143, 1, 288), generator=gen, device=cuda_dev).to(torch.bfloat16)
    pages = []
    for hkv, d, kind in ((1, 128, "bf16"), (2, 64, "e4m3_block"), (1, 64, "e4m3"), (2, 128, "e4m3")):
        plan = _msa().Plan(c.qo, c.kv, 16, hkv, 2, d, 64, 3, c.p, kv_dtype=kind)
        got = c.run(plan)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        pages.append(c.pages.clone())
        plan.latent_append(row[..., :256], row[..., 256:], pages[-1], c.table)
        plan.check_errors()
    assert all(torch.equal(p.view(torch.int16), pages[0].view(torch.int16)) for p in pages[1:])


def test_expand_of_sequences_without_rows(cuda_dev):
    """The pages of all of a plan's sequences are expanded, whether they have new rows or not."""
    rng, kv = np.random.default_rng(2), [10, 300, 129, 256]
    gen = torch.Generator(device=cuda_dev).manual_seed(2)
    rand = lambda *s: torch.randn(s, generator=gen, device=cuda_dev).to(torch.bfloat16)  # noqa: E731
    table, p = _table(kv, 2, rng, cuda_dev)
    c, w_k, w_v = rand(p, 1, 128, 160), rand(3, 96, 128), rand(3, 128, 128)
    _holes(c, table, kv)
    k0, v0 = rand(p, 3, 128, 128), rand(p, 3, 128, 128)
    got = []
    for qo in ([1] * 4, [0, 5, 0, 2]):
        k, v = k0.clone(), v0.clone()
        plan = _msa().Plan(qo, kv, 3, 3, 3, 128, 64, 1, p)
        plan.latent_expand(c, w_k, w_v, table, k, v)
        plan.check_errors()
        got.append((k, v))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and not torch.equal(got[0][0], k0)
