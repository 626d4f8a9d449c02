"""msa_kv_append: scales at the ends of their range."""
import pytest
import torch

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
