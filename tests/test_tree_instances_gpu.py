"""Tree and latent attention through every instance of their kernels (tree_instances.py),
against the definition in 64 bits.  test_launched_kernels_host.py holds the batches to
their instances."""
import gc

import pytest
import torch

from tests import test_latent_gpu, test_tree_attn_gpu
from tests.tree_instances import LATENTS, TREES, batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _collected():
    """Plans that a test's tracebacks hold go with it."""
    yield
    gc.collect()


def _id(x):
    return "-".join(str(v) for v in x) if isinstance(x, tuple) else None


@pytest.mark.parametrize("kind, instance, shape", [
    (kind, *x) for of, kinds in (("bf16", ["bf16"]), ("fp8", ["e4m3", "e4m3_block"])) for x in TREES[of] for kind in kinds], ids=_id)
def test_trees(cuda_dev, kind, instance, shape):
    n, rows, ctx, hq, hkv, hp, topk = shape
    qo, kv = batch(n, rows, ctx)
    for grow in (0.0, 0.4):                               # 0.4: maxima that keep moving
        c = test_tree_attn_gpu.Case(cuda_dev, qo, kv, hq, hkv, hp, instance[3], topk, kind, seed=rows + ctx, grow=grow,
                                    irregular=not grow)
        if grow:
            c.idx_h.sort(-1)
            c.idx = torch.from_numpy(c.idx_h).to(cuda_dev)
        plan = c.plan()
        out, lse = c.run(plan)
        plan.check_errors()
        c.check(out, lse, c.ref())


@pytest.mark.parametrize("instance, shape", LATENTS, ids=_id)
def test_latents(cuda_dev, instance, shape):
    n, rows, ctx, hq, _, hp, topk = shape
    qo, kv = batch(n, rows, ctx)
    for tree, grow, rope in ((False, 0.0, 64), (False, 0.4, 48)) + (((True, 0.0, 16),) if rows <= 128 else ()):
        c = test_latent_gpu.Case(cuda_dev, qo, kv, hq, hp, instance[2], rope, topk, tree, seed=rows + ctx, grow=grow,
                                 irregular=not grow)
        plan = c.plan()
        out, lse = c.run(plan)
        plan.check_errors()
        c.check(out, lse, c.ref())


@pytest.mark.parametrize("latent", [512, 384, 256, 128])
def test_latent_chunk(cuda_dev, latent):
    """A prompt's chunk of several tiles, 64 columns a CTA, no merge."""
    c = test_latent_gpu.Case(cuda_dev, [512, 77], [3000, 900], 32, 1, latent, 64, 9, False, seed=latent)
    plan = c.plan()
    out, lse = c.run(plan)
    plan.check_errors()
    c.check(out, lse, c.ref())
