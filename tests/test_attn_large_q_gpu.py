"""Queries beyond f16 over e4m3 pages: they saturate whichever kernel a row goes
to, so that the rows around it change nothing."""
import numpy as np
import pytest
import torch

from block_sparse_long_proxy_gb300 import synth
from oracle import msa_oracle as O
from tests.gpu_cases import make_plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind, batch, hq", [("e4m3", 2, 16), ("e4m3", 2, 32), ("e4m3", 90, 16), ("e4m3_block", 2, 16),
                                             ("e4m3_block", 90, 32)])
def test_queries_beyond_f16_saturate(cuda_dev, kind, batch, hq):
    """The same row at decode, in a tile of two rows (the decode kernel again, with
    block scales) and in a chunk: one result up to the rounding of weights and
    output.  Anything beyond 65504 is 65504; 65280, which f16 holds, is held to
    the oracle."""
    kv = [300] * batch
    got = {}
    for qo in (1, 2, 150):
        case = synth.Case("large q", [qo] * batch, kv, hq, 2, 128, 2, 64, 3, kv_dtype=kind, page_perm_seed=3)
        inp = synth.make_inputs(case, device=cuda_dev)   # the same pages: they depend on kv_lens and the seed alone
        if qo == 1:
            pages = {n: inp[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale", "kv_indices")}
            # K small, so that logits of such queries stay apart by a few units
            pages["k_scale"] = pages["k_scale"] * 2.0 ** -14
            gen = torch.Generator(device=cuda_dev).manual_seed(1)
            q1 = torch.randn((batch, hq, 128), generator=gen, device=cuda_dev).bfloat16()
        plan = make_plan(case, inp)
        idx = torch.arange(3, dtype=torch.int32, device=cuda_dev).repeat(plan.n_tiles, 2, 1)
        idx[idx >= plan.num_valid_pages[:, None, None]] = -1
        for big in (1e5, -3e38, float("inf"), 65280.0):
            q = inp["q"].clone()
            q.view(batch, qo, hq, 128)[:, -1] = q1
            q[..., 5], q[..., 77] = big, 2.0 * big if abs(big) > 65504 and abs(big) < 1e38 else big
            out, lse = plan.sparse_attn(q, pages["k_pages"], pages["v_pages"], pages["kv_indices"], idx,
                                                        k_scale=pages["k_scale"], v_scale=pages["v_scale"])
            plan.check_errors()
            got[qo, big] = (out.view(batch, qo, hq, 128)[:, -1].double().cpu().numpy(),
                            lse.view(batch, qo, hq)[:, -1].double().cpu().numpy())
            if qo == 1 and big == 65280.0:
                ref, ref_lse = O.sparse_attention(synth.bits(q), synth.bits(pages["k_pages"]), synth.bits(pages["v_pages"]),
                                                  pages["kv_indices"].cpu().numpy(), idx.cpu().numpy(), case.qo_lens, kv,
                                                  k_scale=pages["k_scale"].cpu().numpy(),
                                                  v_scale=pages["v_scale"].cpu().numpy())
                # two of 128 terms are large: sums of products to 2^-12, weights to 2^-10, the output to 2^-8
                assert np.abs(got[1, big][0] - ref).max() <= 2.0 ** -7 * np.abs(ref).max()
                assert np.abs(got[1, big][1] - ref_lse).max() <= 2.0 ** -10 * np.abs(ref_lse).max()
    for (qo, big), (o, l) in got.items():
        assert np.isfinite(o).all() and np.isfinite(l).all()
        assert np.abs(o - got[150, big][0]).max() <= 2.0 ** -7 * np.abs(o).max()
        if big > 0 and big != 65280.0:                   # all of them are 65504
            assert np.array_equal(o, got[qo, 1e5][0]) and np.array_equal(l, got[qo, 1e5][1])
