"""Block-scaled attention over page tables with ids outside the pool: those
blocks are skipped, as if the selection did not name them, and reported; no page
is read in their place."""
import numpy as np
import pytest
import torch

from block_sparse_long_proxy_gb300 import synth
from tests.gpu_cases import make_plan, random_idx

pytestmark = pytest.mark.gpu
_LENS = [int(x) for x in np.random.default_rng(21).integers(200, 3000, size=40)]


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("qo, kv, hq, hkv, topk", [
    ([1] * 5, [700, 129, 1280, 400, 5000], 16, 2, 6), ([1] * 40, _LENS, 64, 4, 9),     # decode, clusters and single CTAs
    ([2] * 20, _LENS[:20], 64, 8, 5),                                                  # tiles of few rows
    ([1] * 9 + [300], _LENS[:10], 48, 4, 6),                                           # beside a chunk
    ([300, 100], [9000, 700], 4, 1, 24),                                               # units over clusters
    ([2000, 300], [2000, 1000], 64, 8, 5)], ids=["decode", "decode many", "few rows", "mixed", "parts", "whole units"])
def test_pages_outside_the_pool_are_skipped(cuda_dev, qo, kv, hq, hkv, topk, d):
    from block_sparse_long_proxy_gb300 import msa
    case = synth.Case("bad", qo, kv, hq, hkv, d, hkv, 64, topk, kv_dtype="e4m3_block", page_perm_seed=3, extra_pages=2)
    inp = synth.make_inputs(case, device=cuda_dev)
    plan = make_plan(case, inp)
    rng = np.random.default_rng(2)
    table = inp["kv_indices"].cpu().numpy()
    # what a page read in place of a bad one would do to any row
    for n in ("k_pages", "v_pages"):
        inp[n].view(torch.uint8)[0] = 0x7E
    inp["v_scale"][0] = 2.0 ** 30
    bad = (rng.random(table.size) < 0.3) | (table == 0)
    ids = np.where(bad, rng.choice([-1, -2 ** 31, plan.num_pages, 2 ** 31 - 1, 2 ** 24], table.size), table).astype(np.int32)
    idx = random_idx(case, rng)
    base = np.concatenate([[0], np.cumsum([(k + 127) // 128 for k in kv])])
    seq = np.repeat(np.arange(len(qo)), [(q + 127) // 128 for q in qo])
    named = np.where(idx < 0, -1, np.where(bad[(base[seq][:, None, None] + np.maximum(idx, 0))], -1, idx)).astype(np.int32)

    def attend(sel, ids, v=inp["v_pages"]):
        return plan.sparse_attn(inp["q"], inp["k_pages"], v, torch.from_numpy(ids).to(cuda_dev),
                                torch.from_numpy(sel).to(cuda_dev), k_scale=inp["k_scale"], v_scale=inp["v_scale"])
    want, want_lse = attend(named, table)
    size, _ = attend(named, table, (inp["v_pages"].view(torch.uint8) & 0x7F).view(torch.float8_e4m3fn))
    plan.check_errors()
    got, lse = attend(idx, ids)
    with pytest.raises(msa.MsaError) as e:
        plan.check_errors()
    assert e.value.status == 6
    # the same sums, in another order where the blocks of a row go to other warps or CTAs: fp32 statistics to 2^-12,
    # weights rounded to f16 on either side (2^-11 of each, so of the sum of weight * |value|), outputs to bf16
    assert torch.equal(torch.isneginf(lse), torch.isneginf(want_lse)) and not torch.isneginf(lse).all()
    fin = torch.isfinite(want_lse)
    assert ((lse - want_lse)[fin].abs() <= 2.0 ** -11 * (1 + want_lse[fin].abs())).all()
    room = 2.0 ** -7 * want.float().abs() + 2.0 ** -9 * size.float()
    assert ((got.float() - want.float()).abs() <= room).all()
    assert (got[~fin] == 0).all()
