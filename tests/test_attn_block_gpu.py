"""Attention over e4m3 pages with one scale for each (page, KV head), prefill
and decode, against the fp64 oracle, and the cache's whole path: rotate,
append, proxy, select, attend.

An output element is a sum of weight * value over the row's keys, divided by
the sum of the probabilities.  Weights are rounded to f16 (2^-11 of each, or
2^-25 absolute below 2^-14, the largest weight of a row being at least 1), the
logits' fp32 sums of 128 products move a probability by 2^-12 at most at these
sizes, and the result is rounded to bf16 (2^-8).  So with A = sum p |v|:
|error| <= 2^-8 |out| + 2^-10 A + keys * 2^-25 * 448 * (largest v_scale)."""
import numpy as np
import pytest
import torch

from block_sparse_long_proxy_gb300 import synth
from oracle import msa_oracle as O
from tests.gpu_cases import compare_out, irregular_idx, make_plan, random_idx

pytestmark = pytest.mark.gpu


def _case(name, qo, kv, hq, hkv, hp, topk, d=128, **kw):
    return synth.Case(name, qo, kv, hq, hkv, d, hp, 64, topk, kv_dtype="e4m3_block", **kw)


def _attend(case, inp, idx, dev, plan=None):
    plan = plan or make_plan(case, inp)
    out, lse = plan.sparse_attn(inp["q"], inp["k_pages"], inp["v_pages"], inp["kv_indices"],
                                torch.from_numpy(idx).to(dev), k_scale=inp["k_scale"], v_scale=inp["v_scale"])
    plan.check_errors()
    return out, lse


def _check(case, inp, idx, out, lse, tile_ids=None):
    args = [synth.bits(inp["q"]), synth.bits(inp["k_pages"]), synth.bits(inp["v_pages"]),
            inp["kv_indices"].cpu().numpy(), idx, case.qo_lens, case.kv_lens]
    kw = dict(k_scale=inp["k_scale"].cpu().numpy(), v_scale=inp["v_scale"].cpu().numpy(), tile_ids=tile_ids)
    o_ref, l_ref = O.sparse_attention(*args, **kw)
    rows = ~np.isnan(o_ref[:, 0, 0])
    args[2] = args[2] & 0x7F
    a_ref, _ = O.sparse_attention(*args, **kw)
    got, gl = out.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
    o_ref, l_ref, a_ref = o_ref[rows], l_ref[rows], a_ref[rows]
    assert np.isfinite(got).all()
    keys = min(case.topk, max((k + 127) // 128 for k in case.kv_lens)) * 128
    tol = 2.0 ** -8 * np.abs(o_ref) + 2.0 ** -10 * a_ref + keys * 2.0 ** -25 * 448 * np.nanmax(kw["v_scale"])
    bad = np.abs(got - o_ref) > tol
    assert not bad.any(), (bad.sum(), np.abs(got - o_ref)[bad].max(), tol[bad].min())
    assert np.array_equal(np.isneginf(gl), np.isneginf(l_ref))
    fin = np.isfinite(l_ref)
    assert (np.abs(gl[fin] - l_ref[fin]) <= 2.0 ** -12 * (1 + np.abs(l_ref[fin]))).all()
    assert (got[np.isneginf(l_ref)] == 0.0).all()


_LENS = [int(x) for x in np.random.default_rng(21).integers(1, 3000, size=40)]
CASES = [
    # decode: split rows and one CTA a row, one and two head tiles, padded selections, one key
    _case("decode one key", [1], [1], 8, 1, 1, 4),
    _case("decode ragged G=8", [1] * 5, [700, 129, 128, 1, 5000], 16, 2, 2, 4, page_perm_seed=2, extra_pages=3),
    _case("decode G=16", [1] * 2, [2048, 777], 32, 2, 2, 5, page_perm_seed=6),
    _case("decode G=3 two block sets a head", [1] * 3, [900, 1500, 33], 12, 2, 4, 6, page_perm_seed=7),
    _case("decode G=1", [1] * 4, [1024, 200, 3000, 129], 3, 3, 3, 3, page_perm_seed=8),
    _case("decode topk 1", [1] * 4, [1024, 200, 3000, 130], 8, 2, 2, 1, page_perm_seed=8),
    _case("decode topk 1024", [1] * 2, [140000, 3000], 8, 1, 1, 1024, page_perm_seed=12),
    _case("decode rows>=SMs", [1] * 20, _LENS[:20], 64, 8, 8, 8, page_perm_seed=9, extra_pages=5),
    _case("decode rows>=SMs G=4 padded", [1] * 40, _LENS, 16, 4, 4, 12, page_perm_seed=10),
    _case("decode rows>=SMs topk 80", [1] * 20, _LENS[:20], 64, 8, 8, 80, page_perm_seed=11),
    _case("decode G=17", [1] * 3, [900, 1500, 33], 34, 2, 2, 6, page_perm_seed=7),
    _case("decode G=40 d64", [1] * 2, [900, 77], 40, 1, 1, 3, d=64, page_perm_seed=7),
    _case("decode rows>=SMs G=16", [1] * 40, _LENS, 64, 4, 4, 5, page_perm_seed=13),
    # prefill
    _case("two rows", [2], [2], 4, 1, 1, 1),
    _case("S=256 G=4", [256], [256], 8, 2, 2, 2),
    _case("ragged chunks", [300, 77, 128, 129], [300, 1000, 128, 500], 8, 2, 2, 3, page_perm_seed=3, extra_pages=5),
    _case("G=1", [256], [256], 2, 2, 2, 2),
    _case("G=3", [200], [333], 6, 2, 2, 2, page_perm_seed=1),
    _case("two block sets a head", [300, 5], [300, 2000], 16, 2, 4, 4, page_perm_seed=1),
    _case("no queries mid-batch", [300, 0, 129], [300, 500, 129], 8, 2, 2, 3, page_perm_seed=6),
    _case("topk 1024", [2048], [2048], 4, 1, 1, 1024, page_perm_seed=7),
    _case("40 blocks", [5120], [5120], 8, 2, 2, 16, page_perm_seed=11),
    # a unit's blocks over clusters of 2, 4 and 8, rows of every part; more parts than some tiles have blocks
    _case("parts 8", [300, 1], [9000, 60], 4, 1, 1, 24, page_perm_seed=3),
    _case("parts 4", [5, 3, 128], [9000, 130, 2000], 12, 4, 4, 9, page_perm_seed=3),
    _case("parts 2", [700], [9000], 12, 4, 4, 9, page_perm_seed=3),
    _case("parts 8 topk 200", [100], [90000], 8, 1, 1, 200, page_perm_seed=3),
    # a short last round, split in a launch of its own
    _case("split tail", [9, 66, 3, 31, 2, 17, 5, 26, 4, 12], [4000, 2100, 1700, 2500, 1999, 60, 1600, 3000, 1920, 130], 32,
          8, 8, 14, page_perm_seed=3),
    # tiles of few rows, several heads side by side: whole groups, odd ones, two sets a KV head, many units
    _case("heads by 16", [2, 1, 8], [900, 1500, 33], 64, 2, 2, 5, page_perm_seed=7),
    _case("heads by 8", [9, 16, 1, 5], [900, 1500, 133, 5], 16, 1, 1, 6, page_perm_seed=7),
    _case("heads by 2, G=3", [33, 64], [900, 1500], 6, 2, 2, 4, page_perm_seed=7),
    _case("heads by 4, G=6", [20, 32, 3], [900, 1500, 300], 12, 1, 2, 4, page_perm_seed=7),
    _case("heads by 8, many units", [int(x) for x in np.random.default_rng(3).integers(1, 10, 40)],
          [int(x) for x in np.random.default_rng(4).integers(10, 900, 40)], 72, 8, 8, 3, page_perm_seed=7),
    _case("d64 heads by 4, G=5", [20, 32, 3], [900, 1500, 300], 5, 1, 1, 4, d=64, page_perm_seed=7),
    # decode rows beside a chunk, and tiles of several kinds of few rows
    _case("mixed batch", [1] * 9 + [300, 1, 20, 64, 7], [900, 1, 2000, 129, 77, 500, 333, 128, 3000, 1100, 700, 20, 64, 900],
          48, 4, 4, 6, page_perm_seed=7, extra_pages=2),
    _case("mixed batch G=3, few units", [200, 1, 65, 4], [900, 700, 1500, 40], 3, 1, 1, 9, page_perm_seed=7),
    _case("mixed batch two sets a head, many units", [1] * 30 + [700], _LENS[:30] + [1500], 64, 2, 4, 5, page_perm_seed=7),
    _case("mixed batch, rows alone", [1, 0, 1, 1], [900, 300, 77, 2000], 16, 2, 2, 6, page_perm_seed=7),
    _case("mixed batch G=16, many rows", [1] * 39 + [40], _LENS[:39] + [90], 64, 4, 4, 9, page_perm_seed=7),
    # tiles of few rows through the decode kernel, in parts of 16 (row, head) columns: one and several parts a tile
    _case("few rows G=8", [2] * 18 + [1, 4, 3], _LENS[:18] + [1, 129, 1500], 64, 8, 8, 5, page_perm_seed=7),
    _case("few rows G=3", [5] * 3 + [6, 2, 1], [900, 5, 133, 2000, 129, 70], 6, 2, 2, 6, page_perm_seed=7),
    _case("few rows G=1", [16] * 3 + [130, 2], [900, 16, 133, 2000, 129], 4, 2, 4, 6, page_perm_seed=7),
    _case("few rows G=16", [3] * 3 + [1], [900, 3, 133, 2000], 16, 1, 1, 6, page_perm_seed=7),
    _case("few rows G=5 d64", [3] * 6 + [200], [900, 3, 133, 2000, 128, 130, 700], 10, 2, 2, 4, d=64, page_perm_seed=7),
    _case("few rows topk 200", [4], [40000], 4, 1, 1, 200, page_perm_seed=7),
    _case("d64 mixed batch", [1] * 5 + [150, 33], [900, 1, 2000, 129, 77, 500, 333], 10, 2, 2, 6, d=64, page_perm_seed=7),
    # head_dim 64
    _case("d64 parts 8", [130], [9000], 6, 1, 2, 24, d=64, page_perm_seed=3),
    _case("d64 decode one key", [1], [1], 8, 1, 1, 4, d=64),
    _case("d64 decode ragged", [1] * 5, [700, 129, 128, 33, 5000], 16, 2, 2, 4, d=64, page_perm_seed=2, extra_pages=3),
    _case("d64 decode G=16", [1] * 3, [2048, 777, 95], 32, 2, 2, 5, d=64, page_perm_seed=6),
    _case("d64 decode rows>=SMs", [1] * 40, _LENS, 32, 4, 4, 12, d=64, page_perm_seed=10),
    _case("d64 decode topk 200", [1] * 2, [30000, 3000], 3, 1, 1, 200, d=64, page_perm_seed=12),
    _case("d64 ragged chunks", [300, 77, 128, 129, 2], [300, 1000, 128, 500, 260], 8, 2, 2, 3, d=64, page_perm_seed=3),
    _case("d64 G=3", [200], [333], 6, 2, 2, 2, d=64, page_perm_seed=1),
    _case("d64 topk 1024", [2048], [2048], 4, 1, 1, 1024, d=64, page_perm_seed=7),
    _case("d64 two block sets a head", [2560], [2600], 16, 2, 4, 9, d=64, page_perm_seed=1),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: c.name)
def test_block_scaled_attention(cuda_dev, case):
    inp = synth.make_inputs(case, device=cuda_dev)
    plan = make_plan(case, inp)
    for seed in (5, 6):                                  # the second call finds the first one's workspace
        idx = random_idx(case, np.random.default_rng(seed))
        out, lse = _attend(case, inp, idx, cuda_dev, plan)
        _check(case, inp, idx, out, lse)
        again, _ = _attend(case, inp, idx, cuda_dev, plan)
        assert torch.equal(out, again)


@pytest.mark.parametrize("qo", [None, 1], ids=["prefill", "decode"])
@pytest.mark.parametrize("rows", [3, 25], ids=["few", "many"])
def test_irregular_selections_and_empty_rows(cuda_dev, qo, rows):
    kv = _LENS[:rows]
    case = _case("irregular", [1] * rows if qo else [min(k, 150) for k in kv], kv, 64, 8, 8, 6, page_perm_seed=4)
    inp = synth.make_inputs(case, device=cuda_dev)
    idx = irregular_idx(case, np.random.default_rng(9))
    out, lse = _attend(case, inp, idx, cuda_dev)
    assert np.isneginf(lse.cpu().numpy()).any()
    _check(case, inp, idx, out, lse)


def test_irregular_selections_in_parts(cuda_dev):
    """The same with few units, whose blocks are shared out over clusters: parts
    without a block, tiles without any."""
    case = _case("irregular parts", [130, 3, 60], [2000, 3, 700], 8, 2, 2, 6, page_perm_seed=4)
    inp = synth.make_inputs(case, device=cuda_dev)
    for seed in (9, 10):
        idx = irregular_idx(case, np.random.default_rng(seed))
        out, lse = _attend(case, inp, idx, cuda_dev)
        assert np.isneginf(lse.cpu().numpy()).any()
        _check(case, inp, idx, out, lse)


@pytest.mark.parametrize("hq, hkv, rows", [(64, 8, 2), (6, 2, 5), (8, 8, 16), (48, 4, 3)])
def test_irregular_selections_few_rows(cuda_dev, hq, hkv, rows):
    """Tiles of few rows, some crossing a page, whose selections leave rows of a
    tile without a key."""
    kv = [max(k, rows) for k in _LENS[:17]] + [129, 130, 256 + rows // 2]
    case = _case("irregular few", [min(rows, 1 + i % rows) for i in range(20)], kv, hq, hkv, hkv, 6, page_perm_seed=4)
    inp = synth.make_inputs(case, device=cuda_dev)
    for seed in (9, 10):
        idx = irregular_idx(case, np.random.default_rng(seed))
        out, lse = _attend(case, inp, idx, cuda_dev)
        assert np.isneginf(lse.cpu().numpy()).any()
        _check(case, inp, idx, out, lse)


@pytest.mark.parametrize("batch", [1, 20])
@pytest.mark.parametrize("decode", [True, False])
def test_scales_far_apart(cuda_dev, decode, batch):
    """Blocks of values 2^50 apart, the softmax's mass on either kind: rows on
    the small block keep its precision.  The keys of block 0 or of block 1 are
    the query itself, so one block holds nearly all of a row's mass."""
    qo, kv = ([1] * batch, [300] * batch) if decode else ([44] * batch, [300] * batch)
    case = _case("far apart", qo, kv, 16, 2, 2, 3, page_perm_seed=1)
    case = case if batch == 1 else _case("far apart", qo, kv, 64, 8, 8, 3, page_perm_seed=1)
    inp = synth.make_inputs(case, device=cuda_dev)
    table = inp["kv_indices"].long().view(batch, 3)
    for heavy in (0, 1):
        for name in ("k_scale", "v_scale"):
            inp[name].fill_(2.0 ** -7)
        inp["v_scale"][table[:, 0]] = 2.0 ** 25 * 1.25
        inp["v_scale"][table[:, 1]] = 2.0 ** -25 * 1.75
        inp["v_scale"][table[:, 2]] = 2.0 ** -25
        # one direction for every query; keys of the heavy block along it, the others against it
        q = torch.full((128,), 1.0, device=cuda_dev)
        inp["q"].copy_(q.to(torch.bfloat16).expand_as(inp["q"]))
        codes = torch.full((3,), -100.0, device=cuda_dev)
        codes[heavy] = 100.0
        k = inp["k_pages"].view(torch.uint8)
        for b in range(3):
            k[table[:, b]] = codes[b].to(torch.float8_e4m3fn).view(torch.uint8)
        idx = np.broadcast_to(np.arange(3, dtype=np.int32), (len(O.tiles_of(qo, kv)), case.hp, 3)).copy()
        out, lse = _attend(case, inp, idx, cuda_dev)
        o_ref, l_ref = O.sparse_attention(synth.bits(inp["q"]), synth.bits(inp["k_pages"]), synth.bits(inp["v_pages"]),
                                          inp["kv_indices"].cpu().numpy(), idx, case.qo_lens, case.kv_lens,
                                          k_scale=inp["k_scale"].cpu().numpy(), v_scale=inp["v_scale"].cpu().numpy())
        got = out.double().cpu().numpy()
        # logits are +-8.8: the light blocks' share is e^-17, so with heavy = 1 the outputs are a mixture of the small
        # block's mean and e^-17 2^50 of the large one's; each weight keeps 2^-10
        args = (synth.bits(inp["q"]), synth.bits(inp["k_pages"]), synth.bits(inp["v_pages"]) & 0x7F,
                inp["kv_indices"].cpu().numpy(), idx, case.qo_lens, case.kv_lens)
        a_ref, _ = O.sparse_attention(*args, k_scale=inp["k_scale"].cpu().numpy(), v_scale=inp["v_scale"].cpu().numpy())
        assert (np.abs(got - o_ref) <= 2.0 ** -8 * np.abs(o_ref) + 2.0 ** -9 * a_ref).all()
        assert np.abs(lse.cpu().numpy() - l_ref).max() <= 2.0 ** -12 * 20


@pytest.mark.parametrize("decode", [True, False])
def test_odd_scales(cuda_dev, decode):
    """Scales that are no powers of two; zero, NaN and infinite ones count as
    the nearer end of [2^-40, 2^40], and those of pages not selected are not
    read."""
    kv = _LENS[:6]
    case = _case("odd", [1] * 6 if decode else [min(k, 200) for k in kv], kv, 8, 2, 2, 4, page_perm_seed=4, extra_pages=2)
    inp = synth.make_inputs(case, device=cuda_dev)
    gen = torch.Generator(device=cuda_dev).manual_seed(3)
    for name in ("k_scale", "v_scale"):
        inp[name] *= 1 + torch.rand(inp[name].shape, generator=gen, device=cuda_dev)
    used = torch.zeros(inp["k_scale"].shape[0], dtype=torch.bool, device=cuda_dev)
    used[inp["kv_indices"].long()] = True
    for name in ("k_scale", "v_scale"):
        inp[name][~used] = float("nan")
    idx = random_idx(case, np.random.default_rng(5))
    out, lse = _attend(case, inp, idx, cuda_dev)
    _check(case, inp, idx, out, lse)
    one = inp["kv_indices"][0].long()
    for v, end in ((0.0, 2.0 ** -40), (float("nan"), 2.0 ** -40), (-1.0, 2.0 ** -40), (float("inf"), 2.0 ** 40)):
        keep = {n: inp[n].clone() for n in ("k_scale", "v_scale")}
        inp["v_scale"][one] = v
        if v != float("inf"):
            inp["k_scale"][one] = v
        a, la = _attend(case, inp, idx, cuda_dev)
        inp["v_scale"][one] = end
        if v != float("inf"):
            inp["k_scale"][one] = end
        b, lb = _attend(case, inp, idx, cuda_dev)
        assert torch.equal(a, b) and torch.equal(la, lb)
        for n, t in keep.items():
            inp[n].copy_(t)


def test_one_scale_everywhere_is_the_static_cache(cuda_dev):
    """With the same scale on every page the cache is the one with a scale a
    head: outputs agree to the rounding of the weights."""
    for qo in ([1] * 3, [300, 20, 129]):
        case = _case("same", qo, [300, 1000, 129], 8, 2, 2, 3, page_perm_seed=3)
        inp = synth.make_inputs(case, device=cuda_dev)
        inp["k_scale"].fill_(0.011)
        inp["v_scale"].fill_(0.007)
        for n in ("k_pages", "v_pages"):                  # the static cache takes no NaN bytes
            raw = inp[n].view(torch.uint8)
            raw[raw == 0x7F] = 0
        idx = random_idx(case, np.random.default_rng(1))
        out, lse = _attend(case, inp, idx, cuda_dev)
        case.kv_dtype = "e4m3"
        st = dict(inp, k_scale=torch.full((2,), 0.011, device=cuda_dev), v_scale=torch.full((2,), 0.007, device=cuda_dev))
        ref, ref_lse = _attend(case, st, idx, cuda_dev)
        assert (out.float() - ref.float()).abs().max() <= 0.007 * 448 * 2.0 ** -7
        assert (lse - ref_lse).abs().max() <= 2.0 ** -12


def test_refusals(cuda_dev):
    from block_sparse_long_proxy_gb300 import msa
    case = _case("refused", [1] * 2, [300, 200], 8, 2, 2, 3)
    inp = synth.make_inputs(case, device=cuda_dev)
    plan = make_plan(case, inp)
    idx = torch.from_numpy(random_idx(case, np.random.default_rng(0))).to(cuda_dev)
    pages = (inp["q"], inp["k_pages"], inp["v_pages"], inp["kv_indices"], idx)
    with pytest.raises(ValueError):
        plan.sparse_attn(*pages, k_scale=inp["k_scale"][0], v_scale=inp["v_scale"][0])
    bad = inp["kv_indices"].clone()
    bad[0] = plan.num_pages
    plan.sparse_attn(inp["q"], inp["k_pages"], inp["v_pages"], bad, idx, k_scale=inp["k_scale"], v_scale=inp["v_scale"])
    with pytest.raises(msa.MsaError) as e:
        plan.check_errors()
    assert e.value.status == 6


def test_checks_mode(cuda_dev, monkeypatch):
    """MSA_CHECKS: bytes behind a sequence's last key raise nothing; a NaN among
    the new rows of an append, or in the queries, does."""
    from block_sparse_long_proxy_gb300 import msa
    monkeypatch.setenv("MSA_CHECKS", "1")
    for qo in ([1] * 2, [150, 3]):
        case = _case("checks", qo, [300, 129], 8, 2, 2, 3)
        inp = synth.make_inputs(case, device=cuda_dev)
        plan = make_plan(case, inp)
        idx = random_idx(case, np.random.default_rng(0))
        _attend(case, inp, idx, cuda_dev, plan)
        k = torch.zeros((sum(qo), 2, 128), device=cuda_dev).bfloat16()
        args = (inp["k_pages"], inp["v_pages"], inp["kv_indices"])
        plan.kv_append(k, k, *args, k_scale=inp["k_scale"], v_scale=inp["v_scale"])
        plan.check_errors()
        bad = k.clone()
        bad[-1, 1, 77] = float("nan")
        for pair in ((bad, k), (k, bad)):
            plan.kv_append(*pair, *args, k_scale=inp["k_scale"], v_scale=inp["v_scale"])
            with pytest.raises(msa.MsaError) as e:
                plan.check_errors()
            assert e.value.status == 7
        plan.kv_append(k, k, *args, k_scale=inp["k_scale"], v_scale=inp["v_scale"])
        inp["q"][0, 0, 0] = float("nan")
        with pytest.raises(msa.MsaError) as e:
            _attend(case, inp, idx, cuda_dev, plan)
        assert e.value.status == 7


def test_captured_decode_step(cuda_dev):
    """Append and attend captured in one graph, replayed over new inputs."""
    case = _case("graph", [1] * 4, [300, 129, 1000, 77], 16, 2, 2, 3, page_perm_seed=3)
    inp = synth.make_inputs(case, device=cuda_dev)
    plan = make_plan(case, inp)
    idx = torch.from_numpy(random_idx(case, np.random.default_rng(1))).to(cuda_dev)
    gen = torch.Generator(device=cuda_dev).manual_seed(3)
    k, v = (torch.randn((4, 2, 128), generator=gen, device=cuda_dev).bfloat16() for _ in range(2))
    out, lse = torch.empty_like(inp["q"]), torch.empty((4, 16), device=cuda_dev)
    cache = {n: inp[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale")}

    def step():
        plan.kv_append(k, v, cache["k_pages"], cache["v_pages"], inp["kv_indices"], k_scale=cache["k_scale"],
                       v_scale=cache["v_scale"])
        plan.sparse_attn(inp["q"], cache["k_pages"], cache["v_pages"], inp["kv_indices"], idx,
                         k_scale=cache["k_scale"], v_scale=cache["v_scale"], out=out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        gen.manual_seed(seed)
        for t in (k, v, inp["q"]):
            t.copy_(torch.randn(t.shape, generator=gen, device=cuda_dev))
        graph.replay()
        got = out.clone(), lse.clone()
        step()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)
        _check(case, inp, idx.cpu().numpy(), out, lse)
    plan.check_errors()


def test_calls_overlap_on_two_streams(cuda_dev):
    """Block-scaled calls use no workspace: two on one plan at once, each the
    result of a call alone."""
    for qo, kv in (([1] * 6, [3000, 129, 1000, 77, 2000, 512]), ([300, 5], [2000, 700]), ([4] * 6, [900] * 6)):
        case = _case("overlap", qo, kv, 32, 2, 2, 12, page_perm_seed=3)
        inp = synth.make_inputs(case, device=cuda_dev)
        plan = make_plan(case, inp)
        idx = torch.from_numpy(random_idx(case, np.random.default_rng(1))).to(cuda_dev)
        kw = dict(k_scale=inp["k_scale"], v_scale=inp["v_scale"])
        qs = [inp["q"], -inp["q"]]
        alone = [plan.sparse_attn(q, inp["k_pages"], inp["v_pages"], inp["kv_indices"], idx, **kw) for q in qs]
        outs = [[(torch.empty_like(q), torch.empty_like(alone[0][1])) for _ in range(8)] for q in qs]
        streams = [torch.cuda.Stream() for _ in qs]
        torch.cuda.synchronize()
        for i in range(8):
            for s, q, o in zip(streams, qs, outs):
                plan.sparse_attn(q, inp["k_pages"], inp["v_pages"], inp["kv_indices"], idx, out=o[i][0], lse=o[i][1],
                                 stream=s, **kw)
        torch.cuda.synchronize()
        plan.check_errors()
        for a, o in zip(alone, outs):
            assert all(torch.equal(a[0], x) and torch.equal(a[1], y) for x, y in o)


@pytest.mark.parametrize("qo, hq", [([1] * 20 + [260], 64), ([700, 3, 80, 500], 12), ([2] * 12, 16)])
def test_steps_back_to_back(cuda_dev, qo, hq):
    """A call's launches overlap each other, never the calls around them: appends
    over the same slots and attention in turn, without a pause and as a graph,
    give what they give one at a time."""
    hkv, n = 4 if hq == 12 else 8, 12
    case = _case("steps", qo, [q + 900 for q in qo], hq, hkv, hkv, 9, page_perm_seed=3)
    inp = synth.make_inputs(case, device=cuda_dev)
    plan = make_plan(case, inp)
    idx = torch.from_numpy(random_idx(case, np.random.default_rng(1))).to(cuda_dev)
    gen = torch.Generator(device=cuda_dev).manual_seed(3)
    new = torch.randn((n, 2, sum(qo), hkv, 128), generator=gen, device=cuda_dev).bfloat16()
    cache = [inp[name] for name in ("k_pages", "v_pages")]
    scales = dict(k_scale=inp["k_scale"], v_scale=inp["v_scale"])
    outs = torch.zeros((n,) + tuple(inp["q"].shape), dtype=torch.bfloat16, device=cuda_dev)
    lse = torch.zeros((n, sum(qo), hq), device=cuda_dev)
    copies = torch.zeros_like(outs)

    def step(i):
        plan.kv_append(new[i, 0], new[i, 1], *cache, inp["kv_indices"], **scales)
        plan.sparse_attn(inp["q"], *cache, inp["kv_indices"], idx, out=outs[i], lse=lse[i], **scales)
        copies[i].copy_(outs[i])
    for i in range(n):
        step(i)
        torch.cuda.synchronize()
    # a page's scale only grows while rows go behind others: the second pass starts where it ended
    for i in range(n):
        step(i)
        torch.cuda.synchronize()
    alone = outs.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(n):
            step(i)
    for run in (lambda: [step(i) for i in range(n)], graph.replay, graph.replay):
        for t in (outs, lse, copies):
            t.zero_()
        run()
        torch.cuda.synchronize()
        assert torch.equal(outs, alone[0]) and torch.equal(lse, alone[1]) and torch.equal(copies, outs)
    plan.check_errors()


@pytest.mark.parametrize("qo", [1, 60])
def test_pages_beyond_4_gib(cuda_dev, qo):
    """The last pages of pools of more than 2^32 bytes: append and attend as on
    small pools, bit for bit, and the first pages stay as they were."""
    kv, hkv, n = [500, 300], 8, 33000                     # 131072 bytes a page
    table = torch.tensor([5, 2, 0, 6, 3, 1, 4], dtype=torch.int32, device=cuda_dev)
    case = _case("far", [qo] * 2, kv, 32, hkv, hkv, 2)
    gen = torch.Generator(device=cuda_dev).manual_seed(5)
    codes = [torch.randint(0, 0x7F, (7, hkv, 128, 128), generator=gen, device=cuda_dev, dtype=torch.uint8) for _ in "kv"]
    new = [torch.randn((2 * qo, hkv, 128), generator=gen, device=cuda_dev).bfloat16() for _ in "kv"]
    q = torch.randn((2 * qo, 32, 128), generator=gen, device=cuda_dev).bfloat16()
    idx = torch.from_numpy(random_idx(case, np.random.default_rng(1))).to(cuda_dev)
    got = []
    for pages in (7, n):
        cache = dict(zip(("k_pages", "v_pages"), (torch.zeros((pages, hkv, 128, 128), dtype=torch.uint8, device=cuda_dev)
                                                  for _ in "kv")))
        cache.update(zip(("k_scale", "v_scale"), (torch.full((pages, hkv), 2.0 ** -6, device=cuda_dev) for _ in "kv")))
        for name, c in zip(("k_pages", "v_pages"), codes):
            cache[name][-7:] = c
            cache[name] = cache[name].view(torch.float8_e4m3fn)
        from block_sparse_long_proxy_gb300 import msa
        plan = msa.Plan([qo] * 2, kv, 32, hkv, hkv, 128, 64, 2, pages, kv_dtype="e4m3_block")
        kv_indices = table + (pages - 7)
        plan.kv_append(*new, cache["k_pages"], cache["v_pages"], kv_indices, k_scale=cache["k_scale"],
                       v_scale=cache["v_scale"])
        got.append(plan.sparse_attn(q, cache["k_pages"], cache["v_pages"], kv_indices, idx, k_scale=cache["k_scale"],
                                    v_scale=cache["v_scale"]))
        plan.check_errors()
        got[-1] += tuple(cache[name][-7:].view(torch.uint8).clone() for name in ("k_pages", "v_pages"))
        if pages > 7:
            assert not any(cache[name].view(torch.uint8)[:7].any().item() for name in ("k_pages", "v_pages"))
        del cache
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_prefill_then_decode_over_the_quantised_cache(cuda_dev):
    """The calls as a server makes them: a ragged prefill and then decode steps,
    queries and keys rotated, K and V appended in e4m3 with block scales, proxy
    keys in bf16 (prefill) and NVFP4 (decode).  Each step's attention agrees
    with the oracle on the cache as it stands, and the whole with attention
    over the unquantised, unpaged keys and values."""
    from block_sparse_long_proxy_gb300 import msa
    dev, hq, hkv, hp, topk = cuda_dev, 16, 2, 2, 64      # topk above every length: the sets are whole
    gen = torch.Generator(device=dev).manual_seed(0)
    rope, pk_rope = msa.Rope(128, base=1e6), msa.Rope(32, layout="interleaved")
    lens = [300, 77, 513]
    table = torch.randperm(20, generator=gen, device=dev).to(torch.int32)
    cap = [4, 2, 6]
    own = [table[:4], table[4:6], table[6:12]]
    u8 = lambda *s: torch.full(s, 0x7F, dtype=torch.uint8, device=dev)  # noqa: E731
    cache = dict(k_pages=u8(20, hkv, 128, 128).view(torch.float8_e4m3fn), v_pages=u8(20, hkv, 128, 128).view(torch.float8_e4m3fn),
                 k_scale=torch.full((20, hkv), float("nan"), device=dev), v_scale=torch.full((20, hkv), float("nan"), device=dev))
    pk_pages = torch.zeros((20, 1, 128, 64), dtype=torch.bfloat16, device=dev)
    fp4 = dict(pk_codes=u8(20, 1, 128, 32), pk_block_scales=u8(20, 1, 128, 4).view(torch.float8_e4m3fn),
               pk_global_scale=torch.full((1,), 6.0 / (448 * 6), device=dev))
    history = [[[], []] for _ in lens]                    # rotated K and V of each sequence, as given
    now = [0, 0, 0]
    for step, qo in enumerate([lens, [1] * 3, [1] * 3, [1] * 3]):
        kv = [a + b for a, b in zip(now, qo)]
        rows = sum(qo)
        nb = [(x + 127) // 128 for x in kv]
        assert all(n <= c for n, c in zip(nb, cap))
        kv_indices = torch.cat([o[:n] for o, n in zip(own, nb)]).contiguous()
        pos = torch.cat([torch.arange(a, b) for a, b in zip(now, kv)]).to(torch.int32).to(dev)
        wide = torch.randn((rows, (hq + 2 * hkv) * 128), generator=gen, device=dev).bfloat16()
        q, k, v = (wide[:, a * 128:b * 128].unflatten(1, (b - a, 128))
                   for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
        pq, pk = (torch.randn((rows, h, 64), generator=gen, device=dev).bfloat16() for h in (hp, 1))
        plan = msa.Plan(qo, kv, hq, hkv, hp, 128, 64, topk, 20, kv_dtype="e4m3_block")
        qr, pqr = rope.apply(q, pos), pk_rope.apply(pq, pos)
        plan.kv_append(k, v, cache["k_pages"], cache["v_pages"], kv_indices, k_scale=cache["k_scale"],
                       v_scale=cache["v_scale"], rope=rope)
        plan.pk_append(pk, kv_indices, pk_pages=pk_pages, rope=pk_rope, **fp4)
        ms = (plan.proxy_maxscore(pqr, pk_pages, kv_indices) if step == 0 else
              plan.proxy_maxscore_nvfp4(pqr, fp4["pk_codes"], fp4["pk_block_scales"], fp4["pk_global_scale"], kv_indices))
        assert torch.isfinite(ms[torch.arange(plan.n_tiles), 0, (plan.num_valid_pages - 1).long()]).all()
        idx = msa.topk_select(ms, topk, plan.num_valid_pages)
        out, lse = plan.sparse_attn(qr, cache["k_pages"], cache["v_pages"], kv_indices, idx, k_scale=cache["k_scale"],
                                    v_scale=cache["v_scale"])
        plan.check_errors()
        case = _case("step", qo, kv, hq, hkv, hp, topk)
        _check(case, dict(cache, q=qr, kv_indices=kv_indices), idx.cpu().numpy(), out, lse)
        # the same attention over what was given
        kr = O.rope(k.double().cpu().numpy(), pos.cpu().numpy(), 128, base=1e6)
        vn, r = v.double().cpu().numpy(), 0
        ref = np.zeros((rows, hq, 128))
        for s, n in enumerate(qo):
            history[s][0].append(kr[r:r + n])
            history[s][1].append(vn[r:r + n])
            ks, vs = (np.concatenate(x) for x in history[s])
            for h in range(hq):
                z = qr[r:r + n, h].double().cpu().numpy() @ ks[:, h // 8].T / np.sqrt(128)
                z = np.where(np.arange(kv[s])[None] <= (now[s] + np.arange(n))[:, None], z, -np.inf)
                w = np.exp(z - z.max(1, keepdims=True))
                ref[r:r + n, h] = (w / w.sum(1, keepdims=True)) @ vs[:, h // 8]
            r += n
        compare_out(out.float().cpu().numpy(), ref, 0.25)     # e4m3: 2^-4 of values up to 4, averaged at the least
        now = kv
