"""The binding's checks of tensors over a library that only answers: host tensors stand
for the device's, device -1 being the current one."""
import os
import subprocess
import sys

import pytest
import torch


class Library:
    """Answers every call with `status` and counts the calls of operators."""

    def __init__(self):
        self.status, self.calls = 0, 0

    def __getattr__(self, name):
        fixed = {"msa_plan": 0, "msa_plan_num_tiles": 2, "msa_plan_max_blocks": 3, "msa_plan_total_q": 5,
                 "msa_plan_num_valid_pages": 0, "msa_last_error": b"refused"}
        if name in fixed:
            return lambda *a: fixed[name]

        def call(*a):
            self.calls += 1
            return self.status
        return call


def stand_in(put):
    """The binding over a Library, by put(object, name, value)."""
    from block_sparse_long_proxy_gb300 import msa
    lib = Library()
    put(msa, "_lib", lib)
    put(msa, "_current_device", lambda: -1)
    put(msa, "_stream", lambda stream=None: None)
    put(msa, "_device_view_int32", lambda *a: None)
    put(torch.cuda, "current_device", lambda: 0)
    return msa, lib


@pytest.fixture
def host(monkeypatch):
    msa, lib = stand_in(monkeypatch.setattr)
    monkeypatch.setattr(msa, "_new", lambda shape, strides, dtype: torch.empty(shape, dtype=dtype))
    return msa, lib


def calls(msa, kind="bf16"):
    """A plan, and each checked call by name: a function of its tensors, and the tensors."""
    plan = msa.Plan([2, 3], [300, 140], 8, 2, 2, 64, 64, 3, 7, kv_dtype=kind)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i4 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kv = (lambda: bf(7, 2, 128, 64)) if kind == "bf16" else (lambda: bf(7, 2, 128, 64).to(torch.float8_e4m3fn))  # noqa: E731
    scale = () if kind == "bf16" else (torch.ones(2), torch.ones(2))
    tree = (bf(5, 8, 64), kv(), kv(), i4(5), i4(2, 2, 3), i4(5, 4)) + scale
    attn = (bf(5, 8, 160), bf(7, 1, 128, 160), i4(5), i4(2, 2, 3), i4(5, 4))
    append = (bf(5, 1, 128), bf(5, 1, 32), bf(7, 1, 128, 160), i4(5))
    expand = (bf(7, 1, 128, 160), bf(2, 32, 128), bf(2, 64, 128), i4(5), bf(7, 2, 128, 64), bf(7, 2, 128, 64))
    table = {"tree_attn": (plan.tree_attn, tree)}
    if kind == "bf16":
        table |= {"latent_attn": (lambda *t: plan.latent_attn(*t[:4], 32, 0.1, tree_mask=t[4]), attn),
                  "latent_append": (plan.latent_append, append), "latent_expand": (plan.latent_expand, expand)}
    return plan, table


@pytest.mark.parametrize("name", ["tree_attn", "latent_attn", "latent_append", "latent_expand"])
def test_refused_calls_leave_no_record(host, monkeypatch, name):
    """Tensors of a call that the library refused (the plan is another device's, for one) are
    checked again: what a record says of their device holds for accepted calls only."""
    msa, lib = host
    plan, table = calls(msa)
    fn, tensors = table[name]
    lib.status = 1
    for _ in range(2):
        with pytest.raises(msa.MsaError):
            fn(*tensors)
    assert not plan._alike
    lib.status, before = 0, lib.calls
    monkeypatch.setattr(msa, "_current_device", lambda: 0)  # the plan's; the tensors are elsewhere
    with pytest.raises(ValueError):
        fn(*tensors)
    assert lib.calls == before
    monkeypatch.setattr(msa, "_current_device", lambda: -1)
    for _ in range(3):
        fn(*tensors)
    assert lib.calls == before + 3


@pytest.mark.parametrize("name, kind, pair", [("tree_attn", "e4m3", (6, 7)), ("tree_attn", "bf16", (1, 2)),
                                              ("latent_append", "bf16", (0, 1))])
def test_one_tensor_twice(host, monkeypatch, name, kind, pair):
    """A comparison of a call that has one tensor in two places never passes: none is made for it,
    call after call, nor taken from another call's place."""
    msa, lib = host
    made, real = [], msa._Alike

    def alike(*tensors, **kw):
        made.append(len(tensors))
        return real(*tensors, **kw)
    monkeypatch.setattr(msa, "_Alike", alike)
    plan, table = calls(msa, kind)
    fn, tensors = table[name]
    if name == "latent_append":                           # as wide as each other
        tensors = (tensors[0][..., :32].contiguous(), tensors[1], torch.zeros((7, 1, 128, 64), dtype=torch.bfloat16), tensors[3])
    args = (lambda t: fn(*t[:6], k_scale=t[6], v_scale=t[7])) if kind == "e4m3" else (lambda t: fn(*t))  # noqa: E731
    twice = list(tensors)
    twice[pair[1]] = twice[pair[0]]
    for _ in range(3):
        args(twice)
    assert made == [] and lib.calls == 3
    for _ in range(3):
        args(tensors)
        args(twice)
    assert len(made) == 1 and lib.calls == 9


MISSING = """
import torch
from torch._C._dynamo import guards
%s
import tests.test_binding_host as t
msa, lib = t.stand_in(setattr)
empty, devices = torch.empty, []
def on_host(shape, dtype, device):
    devices.append(device)
    return empty(shape, dtype=dtype)
torch.empty = on_host
plan, table = t.calls(msa)
for name, (fn, tensors) in table.items():
    got = [fn(*tensors) for _ in range(3)]
    if name in ("tree_attn", "latent_attn"):
        for out, lse in got:
            wide = 64 if name == "tree_attn" else 128
            assert out.shape == (5, 8, wide) and out.dtype is torch.bfloat16 and out.is_contiguous()
            assert lse.shape == (5, 8) and lse.dtype is torch.float32 and lse.is_contiguous()
assert lib.calls == 12 and not plan._alike and devices == ["cuda"] * 12, (plan._alike, devices)
"""


@pytest.mark.parametrize("change", ["del guards._empty_strided_cuda, guards.TensorGuards", "del torch._C._dynamo",
                                    "del guards._empty_strided_cuda\nguards.TensorGuards = lambda *a: None"],
                         ids=["without either name", "without the module", "another constructor"])
def test_torch_without_private_parts(change):
    """What the binding takes of torch beyond its public names saves time only: without it every
    call makes all checks and its outputs by torch.empty."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", MISSING % change], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
