"""How far block-scaled attention may be off, row by row, for long selections too.

Against fp64, per row and head over the head's dims (norms).  p_k are the row's
probabilities, v_k its values, c_k their codes and s_k their scales:
  - the output is rounded to bf16: 2^-8 |out|;
  - each weight is rounded to f16, by 2^-11 of itself at most, and the errors of
    different keys add as independent ones do: |sum p_k d_k v_k| with |d_k| <=
    2^-11 is within 4 * 2^-11 S, S^2 = sum p_k^2 v_k^2 over keys and dims (seven
    standard deviations of a rounding error).  Where many keys have one weight
    they share its error: 2^-11 |out|;
  - a weight below 2^-14 is off by 2^-25 instead, the largest weight of a row
    being 1 at least: 4 * 2^-25 max(p_k s_k) |c|, |c|^2 the sum of c_k^2;
  - fp32 logits and sums: below 2^-12 |out| at these sizes.
The bound is checked to be one that an output 5 % off does not pass."""
import numpy as np
import pytest
import torch

from block_sparse_long_proxy_gb300 import synth
from oracle import msa_oracle as O
from tests.gpu_cases import make_plan, random_idx
from tests.test_attn_block_gpu import CASES

pytestmark = pytest.mark.gpu


def _reference(case, inp, idx, tile_ids):
    """For each (row, head) of the tiles: out, lse and the bound on |got - out|."""
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    q, k, v = f(inp["q"]), *(O.e4m3_to_f64(inp[n].view(torch.uint8).cpu().numpy()) for n in ("k_pages", "v_pages"))
    ks, vs = f(inp["k_scale"]), f(inp["v_scale"])
    table, indptr = inp["kv_indices"].cpu().numpy(), O.kv_indptr(case.kv_lens)
    tiles, grp, per_kv = O.tiles_of(case.qo_lens, case.kv_lens), case.hq // case.hp, case.hp // case.hkv
    rows, out, lse, tol = [], [], [], []
    for t in tile_ids:
        tl = tiles[t]
        n = tl.q_end - tl.q_begin
        pos = tl.pos0 + np.arange(n)
        o, l, b = np.zeros((n, case.hq, case.d)), np.full((n, case.hq), -np.inf), np.zeros((n, case.hq))
        for p in range(case.hp):
            sel = np.array(sorted(j for j in idx[t, p] if j >= 0), dtype=np.int64)
            if not len(sel):
                continue
            page, g = table[indptr[tl.seq] + sel], p // per_kv
            keys = (sel[:, None] * 128 + np.arange(128)).ravel()
            seen = keys <= pos[-1]                       # the others are behind the tile's last row
            keys = keys[seen]
            s_k, s_v = (np.repeat(x[page, g], 128)[seen] for x in (ks, vs))
            kc, vc = (x[page, g].reshape(-1, case.d)[seen] for x in (k, v))
            for h in range(p * grp, (p + 1) * grp):
                z = q[tl.q_begin:tl.q_end, h] @ kc.T * s_k / np.sqrt(case.d)
                z = np.where(keys[None] <= pos[:, None], z, -np.inf)
                some = np.isfinite(z).any(1)
                top = np.where(some, z.max(1), 0.0)
                w = np.exp(z - top[:, None])
                total = w.sum(1)
                l[some, h] = (top + np.log(np.maximum(total, 1e-300)))[some]
                pr = np.where(some[:, None], w / np.maximum(total, 1e-300)[:, None], 0.0)
                val, c2 = vc * s_v[:, None], (vc ** 2).sum(1)
                o[:, h] = pr @ val
                spread = np.sqrt((pr ** 2) @ (c2 * s_v ** 2))
                small = (pr * s_v).max(1) * np.sqrt((keys[None] <= pos[:, None]) @ c2)
                b[:, h] = ((2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12) * np.linalg.norm(o[:, h], axis=1) + 2.0 ** -9 * spread
                           + 2.0 ** -23 * small)
        rows.append(np.arange(tl.q_begin, tl.q_end))
        out.append(o), lse.append(l), tol.append(b)
    return tuple(np.concatenate(x) for x in (rows, out, lse, tol))


@pytest.mark.parametrize("case", CASES, ids=lambda c: c.name)
def test_error_of_each_row(cuda_dev, case):
    inp = synth.make_inputs(case, device=cuda_dev)
    plan = make_plan(case, inp)
    idx = random_idx(case, np.random.default_rng(8))
    out, lse = plan.sparse_attn(inp["q"], inp["k_pages"], inp["v_pages"], inp["kv_indices"],
                                torch.from_numpy(idx).to(cuda_dev), k_scale=inp["k_scale"], v_scale=inp["v_scale"])
    plan.check_errors()
    n = plan.n_tiles
    tile_ids = sorted({0, 1 % n, n // 3, n // 2, n - 2 if n > 1 else 0, n - 1})
    rows, ref, ref_lse, tol = _reference(case, inp, idx, tile_ids)
    size = np.linalg.norm(ref, axis=-1)
    seen = np.isfinite(ref_lse)
    assert (tol[seen] < 0.05 * size[seen]).all()
    err = np.linalg.norm(out.double().cpu().numpy()[rows] - ref, axis=-1)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()
    got = lse.double().cpu().numpy()[rows]
    assert np.array_equal(np.isfinite(got), seen)
    assert (np.abs(got[seen] - ref_lse[seen]) <= 2.0 ** -12 * (1 + np.abs(ref_lse[seen]))).all()
