"""Tensors over a plan's device tables."""
import gc

import numpy as np
import pytest

from oracle import msa_oracle as O

pytestmark = pytest.mark.gpu


def test_a_view_keeps_its_plan(cuda_dev, monkeypatch):
    """num_valid_pages may outlive the Plan that it came from: the tables stay
    until the last view is gone, and then go."""
    from block_sparse_long_proxy_gb300 import msa
    destroyed, destroy = [], msa._lib.msa_plan_destroy
    monkeypatch.setattr(msa._lib, "msa_plan_destroy", lambda h: destroyed.append(h.value))
    qo, kv = [300, 5], [700, 130]
    plan = msa.Plan(qo, kv, 8, 2, 2, 128, 64, 3, num_pages=8)
    at = plan._h.value
    part = plan.num_valid_pages[1:]
    del plan
    gc.collect()
    assert destroyed == []
    assert np.array_equal(part.cpu().numpy(), O.num_valid_pages(qo, kv)[1:])
    del part
    gc.collect()
    assert destroyed == [at]
    destroy(at)
