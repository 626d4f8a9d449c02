"""YaRN where its ramp would begin before the first pair or end behind the last."""
import numpy as np
import pytest
import torch

from oracle import msa_oracle as O

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw, rot, lo, hi", [
    (dict(original_len=128, beta_fast=32.0), 64, -2, 11),            # no pair turns 32 times
    (dict(original_len=10 ** 6, beta_slow=0.002), 64, 29, 64),       # all turn more often than 0.002 times
    (dict(original_len=128, base=1.5, beta_fast=4.0, beta_slow=0.001), 16, 32, 196),   # both
    (dict(original_len=4096, beta_fast=8.0, beta_slow=8.0), 64, 15, 16)], ids=str)
def test_ramp_kept_within_the_pairs(cuda_dev, kw, rot, lo, hi):
    """The published clamps: the ramp runs from max(floor D(beta_fast), 0) to
    min(ceil D(beta_slow), rotary_dim - 1)."""
    from block_sparse_long_proxy_gb300 import msa
    base = kw.get("base", 10000.0)
    turning = lambda b: rot * np.log(kw["original_len"] / (2 * np.pi * b)) / (2 * np.log(base))  # noqa: E731
    assert (int(np.floor(turning(kw.get("beta_fast", 32.0)))), int(np.ceil(turning(kw.get("beta_slow", 1.0))))) == (lo, hi)
    i = np.arange(rot // 2)
    lo, hi = max(lo, 0), min(hi, rot - 1)
    ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
    f = base ** (-2.0 * i / rot)
    f = f * (1 - ramp) + f / 5.0 * ramp
    assert np.allclose(f, O.rope_freqs(rot, scaling="yarn", factor=5.0, **kw)[0], rtol=1e-14)
    pos = np.array([0, 1, 100, 4097, 131071, -3], dtype=np.int32)
    x = torch.randn((6, 2, rot), generator=torch.Generator(device=cuda_dev).manual_seed(1), device=cuda_dev)
    got = msa.Rope(rot, scaling="yarn", factor=5.0, **kw).apply(x, torch.from_numpy(pos).to(cuda_dev)).double().cpu().numpy()
    a, b = (y.double().cpu().numpy() for y in (x[..., :rot // 2], x[..., rot // 2:]))
    m, t = 0.1 * np.log(5.0) + 1.0, (np.outer(pos, f) % (2 * np.pi))[:, None]
    want = m * np.concatenate((a * np.cos(t) - b * np.sin(t), b * np.cos(t) + a * np.sin(t)), axis=-1)
    # angles, cos and sin, the factor, two products and a sum: below 2^-21 of |a| + |b|
    room = 2.0 ** -21 * m * (np.abs(a) + np.abs(b))
    assert (np.abs(got - want) <= np.concatenate((room, room), axis=-1)).all()
