"""msa_kv_append: scales at the ends of their range, several heads a CTA."""
import numpy as np
import pytest
import torch

from oracle import msa_oracle as O
from tests.test_cache_ops_gpu import BF16, ROT, _codes_between, _f64, _fresh_codes, _partner_sum

pytestmark = pytest.mark.gpu


def _mean_value(msa, pages, scales, table, kv, dev):
    """The mean of a sequence's values as the attention has them: a query of zeros."""
    plan = msa.Plan([1], [kv], 1, 1, 1, 128, 64, 1, pages[0].shape[0], kv_dtype="e4m3_block")
    q, idx = torch.zeros((1, 1, 128), device=dev).bfloat16(), torch.zeros((1, 1, 1), dtype=torch.int32, device=dev)
    out, _ = plan.sparse_attn(q, *pages, table, idx, k_scale=scales[0], v_scale=scales[1])
    plan.check_errors()
    return out.float()


@pytest.mark.parametrize("old", [2.0 ** -50, 1e-30, 1e-42, 2.0 ** -40])
def test_scales_below_the_least(cuda_dev, old):
    """A page whose scale lies below 2^-40 holds, to the attention, codes of 2^-40:
    an append behind them leaves them that, or converts them from it."""
    from block_sparse_long_proxy_gb300 import msa
    table = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    codes = torch.arange(2 * 5 * 128, device=cuda_dev).remainder(0x7F).to(torch.uint8).view(2, 1, 1, 5, 128)
    for new, factor in ((0.0, 1.0), (448 * 2.0 ** -38, 0.25)):
        pages = torch.zeros((2, 1, 1, 128, 128), dtype=torch.uint8, device=cuda_dev)
        pages[..., :5, :] = codes
        pages = [p.view(torch.float8_e4m3fn) for p in pages]
        scales = [torch.full((1, 1), old, device=cuda_dev) for _ in "kv"]
        before = _mean_value(msa, pages, scales, table, 5, cuda_dev)
        plan = msa.Plan([1], [6], 1, 1, 1, 128, 64, 1, 1, kv_dtype="e4m3_block")
        row = torch.full((1, 1, 128), new, device=cuda_dev).bfloat16()
        plan.kv_append(row, row, *pages, table, k_scale=scales[0], v_scale=scales[1])
        plan.check_errors()
        for p, s, c in zip(pages, scales, codes):
            assert float(s) == 2.0 ** -40 / factor
            want = (c[0, 0].view(torch.float8_e4m3fn).float() * factor).to(torch.float8_e4m3fn)
            assert torch.equal(p[0, 0, :5].view(torch.uint8), want.view(torch.uint8))
        # exact but for the codes below e4m3's smallest step, half of which (2^-10 of the new scale) is the most lost
        after = _mean_value(msa, pages, scales, table, 5, cuda_dev)
        assert ((after - before).abs() <= 2.0 ** -7 * before.abs() + 2.0 ** -10 * 2.0 ** -40 / factor).all()


# 260 pages that get rows: enough for eight heads a CTA (K; four of V)
def _many_pages():
    rng = np.random.default_rng(12)
    new = [int(x) for x in rng.integers(1, 11, 200)] + [int(x) for x in rng.integers(130, 300, 20)]
    before = [int(x) for x in rng.integers(0, 128, 220)]
    before[::7] = [0] * len(before[::7])                 # pages that start anew
    return new, [a + b for a, b in zip(new, before)]


@pytest.mark.parametrize("hkv, d, rot, layout", [(8, 128, 128, "half"), (7, 128, 96, "interleaved"), (3, 128, 64, "half"),
                                                 (12, 64, 64, "interleaved")])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3_block"])
def test_several_heads_a_cta(cuda_dev, kind, hkv, d, rot, layout):
    """Every head of every page as the definition has it, where a CTA takes several:
    all heads, a last group of fewer, pages partly filled and anew, infinities among
    some heads' rows."""
    from block_sparse_long_proxy_gb300 import msa
    qo, kv = _many_pages()
    rows, nb = sum(qo), [(k + 127) // 128 for k in kv]
    units = sum((k + 127) // 128 - (k - q) // 128 for q, k in zip(qo, kv))
    assert units * 2 >= 3 * torch.cuda.get_device_properties(cuda_dev).multi_processor_count
    gen = torch.Generator(device=cuda_dev).manual_seed(hkv)
    p = sum(nb) + 2
    table = torch.randperm(p, generator=gen, device=cuda_dev)[:sum(nb)].to(torch.int32)
    x = [(torch.randn((rows, hkv, d), generator=gen, device=cuda_dev)
          * torch.exp(torch.randn((rows, 1, 1), generator=gen, device=cuda_dev))).to(torch.bfloat16) for _ in "kv"]
    if kind == "e4m3_block":                             # in dims that do not turn
        for t, dims in ((x[0], range(rot, d)), (x[1], range(d))):
            for i in range(0, rows, 37) if len(dims) else ():
                t[i, i % hkv, dims[i % len(dims)]] = float("inf") if i % 2 else float("-inf")
    shape = (p, hkv, 128, d)
    if kind == "bf16":
        pages, scales = [torch.randn(shape, generator=gen, device=cuda_dev).to(torch.bfloat16) for _ in "kv"], [None] * 2
    else:
        pages = [_fresh_codes(shape, gen, cuda_dev) for _ in "kv"]
        scales = [torch.rand(hkv, generator=gen, device=cuda_dev) * 0.02 + 0.002 if kind == "e4m3" else
                  torch.exp2(torch.randint(-12, 0, (p, hkv), generator=gen, device=cuda_dev).float()) for _ in "kv"]
    before = [t.clone() for t in pages]
    old = [None if s is None else _f64(s) for s in scales]
    plan = msa.Plan(qo, kv, hkv, hkv, hkv, d, 32, 1, p, kv_dtype=kind)
    plan.kv_append(*x, *pages, table, k_scale=scales[0], v_scale=scales[1], rope=msa.Rope(rot, layout))
    plan.check_errors()
    at, pos = table.cpu().numpy(), np.concatenate([np.arange(b - a, b) for a, b in zip(qo, kv)])
    for t, got, b, s, o, turned in zip(x, pages, before, scales, old, (True, False)):
        ref = O.rope(_f64(t), pos, rot, layout) if turned else _f64(t)
        delta = ROT * _partner_sum(_f64(t), rot, layout) if turned else np.zeros(ref.shape)
        # where the rows went: their values and the distances, NaN elsewhere
        where, _ = O.kv_append(ref, np.full(shape, np.nan), at, qo, kv, "bf16")
        dl, _ = O.kv_append(delta, np.zeros(shape), at, qo, kv, "bf16")
        new = ~np.isnan(where)
        if kind == "bf16":
            assert np.array_equal(_f64(got)[~new], _f64(b)[~new])
            room = dl + BF16 * (np.abs(where) + dl) * turned
            assert (np.abs(_f64(got) - where)[new] <= room[new]).all()
            continue
        code, raw = got.view(torch.uint8).cpu().numpy(), b.view(torch.uint8).cpu().numpy()
        if kind == "e4m3":
            assert np.array_equal(code[~new], raw[~new])
            by = np.broadcast_to(_f64(s)[None, :, None, None], shape)
            _codes_between(code[new], where[new], (dl + np.abs(where) * 2.0 ** -24)[new], by[new])
            continue
        want, want_s = O.kv_append(ref, raw, at, qo, kv, kind, o)
        if not turned:
            assert np.array_equal(_f64(s), want_s) and np.array_equal(code, want)
            continue
        # a page's largest value may lie within delta of a border between scales
        same = np.broadcast_to((_f64(s) == want_s)[:, :, None, None], shape)
        assert same.mean() > 0.99
        assert np.array_equal(code[~new & same], want[~new & same])
        by = np.broadcast_to(_f64(s)[:, :, None, None], shape)
        fin = new & same & np.isfinite(where)
        _codes_between(code[fin], where[fin], dl[fin], by[fin])
        assert np.array_equal(code[new & np.isinf(where)], want[new & np.isinf(where)])
