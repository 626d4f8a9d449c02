"""Rotary angles at positions up to the ends of int32, against frequencies and
angles of 60 decimal digits.

Rotating (1, 0) gives (m cos t, m sin t).  The table's fraction of a turn is off
by 2^-65 turns at most, the phase at 2^31 by 2^-34; the polynomials leave out
terms below 2^-28 and round what is left of them below 2^-27, and their sum is
rounded to the nearest fp32: half a step of the value and 2^-26 m in all."""
import math
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def _turns(rot, base, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """Turns a position of each pair, as Decimals, and the factor m."""
    b, f, one, out = Decimal(base), Decimal(factor), Decimal(1), []
    if scaling == "ntk":
        b = b * f ** (Decimal(rot) / (rot - 2))
    if scaling == "yarn":
        def pair(times):
            return rot * math.log(original_len / (2 * math.pi * times)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot - 1)
    for i in range(rot // 2):
        t = b ** (Decimal(-2 * i) / rot) / (2 * PI)
        if scaling == "linear":
            t = t / f
        if scaling == "yarn":
            r = min(max(Decimal(i - lo) / max(hi - lo, Decimal("0.001")), Decimal(0)), one)
            t = t * (one - r) + t / f * r
        out.append(t)
    return out, 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1 else 1.0


@pytest.mark.parametrize("rot, layout, base, scaling", [
    (64, "half", 10000.0, {}), (128, "interleaved", 500000.0, {}), (16, "half", 1.5, dict(scaling="linear", factor=3.7)),
    (64, "half", 10000.0, dict(scaling="ntk", factor=8.3)),
    (128, "interleaved", 1e6, dict(scaling="yarn", factor=5.3, original_len=4096))])
def test_angles_at_far_positions(cuda_dev, rot, layout, base, scaling):
    from block_sparse_long_proxy_gb300 import msa
    pos = [2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31, -2 ** 31 + 77, 2 ** 30 + 12345, 1987654321, -1234567890, 2 ** 24 + 1, 131071, 0]
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    x = torch.zeros((len(pos), 1, rot), device=cuda_dev)
    x[..., a] = 1.0
    p = torch.tensor(pos, dtype=torch.int32, device=cuda_dev)
    rope = msa.Rope(rot, layout, base=base, **scaling)
    got, back = (rope.apply(x, p, inverse=inv).double().cpu().numpy()[:, 0] for inv in (False, True))
    ref = np.zeros((len(pos), rot // 2))
    with localcontext() as ctx:
        ctx.prec = 60
        turns, m = _turns(rot, base, **scaling)
        for i, n in enumerate(pos):
            for j, t in enumerate(turns):
                turn = n * t
                ref[i, j] = float(turn - turn.to_integral_value())
    c, s = m * np.cos(2 * np.pi * ref), m * np.sin(2 * np.pi * ref)
    for out, want in ((got[:, a], c), (got[:, b], s), (back[:, a], c), (back[:, b], -s)):
        tol = np.spacing(np.abs(want).astype(np.float32)).astype(np.float64) / 2 + 2.0 ** -26 * m
        assert (np.abs(out - want) <= tol).all(), np.abs(out - want).max()
