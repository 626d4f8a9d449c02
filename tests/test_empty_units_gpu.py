"""Prefills whose selections leave many (tile, group) rows without a block, over
many units a CTA: the units without work go through the same barriers as the
others, in whatever order the kernel's warps come to them."""
import numpy as np
import pytest
import torch

from block_sparse_long_proxy_gb300 import synth
from tests.gpu_cases import make_plan, random_idx

pytestmark = pytest.mark.gpu


def _emptied(idx, pattern, rng):
    """Rows of a selection emptied: all, two of three in turn, or at random."""
    idx = idx.copy()
    n = idx.shape[0] * idx.shape[1]
    drop = dict(all=np.ones(n, bool), runs=np.arange(n) % 3 > 0, random=rng.random(n) < 0.6)[pattern]
    idx.reshape(n, -1)[drop] = -1
    return idx, drop.reshape(idx.shape[:2])


@pytest.mark.parametrize("pattern", ["all", "runs", "random"])
@pytest.mark.parametrize("kind, d, hq", [("bf16", 128, 24), ("bf16", 64, 24), ("e4m3", 128, 24), ("e4m3_block", 128, 24),
                                         ("e4m3_block", 64, 24), ("e4m3_block", 128, 40)])
def test_units_without_blocks(cuda_dev, kind, d, hq, pattern):
    """A row's result does not depend on the rows around it: it has the bits of
    the call whose rows all have blocks, or is 0 (lse -inf)."""
    case = synth.Case("empty", [4000, 90, 20], [4000, 2000, 500], hq, 8, d, 8, 64, 3, kv_dtype=kind)
    inp = synth.make_inputs(case, device=cuda_dev)
    plan = make_plan(case, inp)
    rng = np.random.default_rng(4)
    full = random_idx(case, rng)
    scales = {} if kind == "bf16" else {n: inp[n] for n in ("k_scale", "v_scale")}

    def attend(idx, out=None, lse=None):
        return plan.sparse_attn(inp["q"], inp["k_pages"], inp["v_pages"], inp["kv_indices"],
                                torch.from_numpy(idx).to(cuda_dev), out=out, lse=lse, **scales)
    whole, whole_lse = attend(full)
    plan.check_errors()
    out, lse = torch.empty_like(whole), torch.empty_like(whole_lse)
    for _ in range(40):
        idx, drop = _emptied(full, pattern, rng)
        tile = np.repeat(np.arange(plan.n_tiles), [min(128, q - t) for q in case.qo_lens for t in range(0, q, 128)])
        gone = torch.from_numpy(drop[tile].repeat(hq // 8, axis=1)).to(cuda_dev)
        attend(idx, out, lse)
        plan.check_errors()
        assert torch.equal(lse, whole_lse.masked_fill(gone, float("-inf")))
        assert torch.equal(out, whole.masked_fill(gone[..., None], 0.0))


@pytest.mark.parametrize("pattern", ["all", "random"])
def test_units_without_blocks_backward(cuda_dev, pattern):
    """The backward's proxy softmax has such units, too."""
    case = synth.Case("empty", [4000, 90], [4000, 2000], 16, 8, 128, 8, 64, 3)
    inp = synth.make_inputs(case, device=cuda_dev, with_dout=True)
    plan = make_plan(case, inp)
    rng = np.random.default_rng(4)
    idx, drop = _emptied(random_idx(case, rng), pattern, rng)
    idx = torch.from_numpy(idx).to(cuda_dev)
    pages = (inp["k_pages"], inp["v_pages"], inp["kv_indices"], idx)
    out, lse = plan.sparse_attn(inp["q"], *pages)
    first = None
    for _ in range(10):
        grads = plan.sparse_attn_bwd(inp["q"], *pages, out, lse, inp["dout"], inp["pq"], inp["pk_pages"])
        plan.check_errors()
        first = first or grads
        assert all(torch.equal(grads[n], first[n]) for n in grads)
    tile = np.repeat(np.arange(plan.n_tiles), [min(128, q - t) for q in case.qo_lens for t in range(0, q, 128)])
    gone = torch.from_numpy(drop[tile]).to(cuda_dev)
    assert (first["dpq"][gone] == 0).all() and (first["dq"][gone.repeat_interleave(2, 1)] == 0).all()
    assert pattern == "all" or first["dpq"][~gone].abs().sum() > 0
