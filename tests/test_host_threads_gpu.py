"""Calls from host threads other than the one that made the plan, and from several
at once."""
import threading

import numpy as np
import pytest
import torch

from block_sparse_long_proxy_gb300 import synth
from tests.gpu_cases import make_plan, random_idx

pytestmark = pytest.mark.gpu


def _on_threads(workers, times=1):
    """workers: functions of a stream.  Each `times` times on a new thread of its
    own, all at once; the first exception of any is raised."""
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(workers)), []
    streams = [torch.cuda.Stream() for _ in workers]

    def loop(fn, stream):
        try:
            start.wait()
            for _ in range(times):
                fn(stream)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=loop, args=a) for a in zip(workers, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if failed:
        raise failed[0]


@pytest.mark.parametrize("kind, qo", [("bf16", 200), ("e4m3", 200), ("e4m3", 1), ("e4m3_block", 200), ("e4m3_block", 1)])
def test_first_call_of_a_thread(cuda_dev, kind, qo):
    """A new thread has no CUDA context until a call of it makes one current:
    whichever call of the library comes first there works."""
    case = synth.Case("thread", [qo] * 2, [300, 700], 16, 2, 128, 2, 64, 3, kv_dtype=kind)
    inp = synth.make_inputs(case, device=cuda_dev)
    plan = make_plan(case, inp)
    idx = torch.from_numpy(random_idx(case, np.random.default_rng(1))).to(cuda_dev)
    scales = {} if kind == "bf16" else {n: inp[n] for n in ("k_scale", "v_scale")}

    def attend(stream=None, **out):
        return plan.sparse_attn(inp["q"], inp["k_pages"], inp["v_pages"], inp["kv_indices"], idx, stream=stream,
                                **scales, **out)

    def score(stream=None, out=None):
        return plan.proxy_maxscore(inp["pq"], inp["pk_pages"], inp["kv_indices"], out=out, stream=stream)
    want, ms = attend(), score()
    out, lse, ms2 = (torch.empty_like(t) for t in (*want, ms))
    _on_threads([lambda s: attend(s, out=out, lse=lse)])
    _on_threads([lambda s: score(s, out=ms2)])
    plan.check_errors()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(ms2, ms)


# Two threads at once, each with a plan, stream and cache of its own: what one
# thread's calls ask of the CUDA runtime leaves the other's alone.

@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3_block"])
def test_decode_and_prefill_appends_at_once(cuda_dev, kind):
    workers, got, want, plans = [], [], [], []
    for qo, kv in (([1] * 4, [300, 129, 1000, 77]), ([150, 20], [300, 20])):
        case = synth.Case("at once", qo, kv, 16, 2, 128, 2, 64, 3, kv_dtype=kind)
        inp = synth.make_inputs(case, device=cuda_dev)
        plans.append(make_plan(case, inp))
        gen = torch.Generator(device=cuda_dev).manual_seed(3)
        k, v = (torch.randn((case.total_q, 2, 128), generator=gen, device=cuda_dev).bfloat16() for _ in range(2))

        def append(cache, stream=None, plan=plans[-1], k=k, v=v, table=inp["kv_indices"]):
            plan.kv_append(k, v, kv_indices=table, stream=stream, **cache)
        names = ("k_pages", "v_pages") + (() if kind == "bf16" else ("k_scale", "v_scale"))
        alone, shared = ({n: inp[n].clone() for n in names} for _ in range(2))
        append(alone)
        plans[-1].check_errors()
        workers.append(lambda s, append=append, cache=shared: append(cache, s))
        got.append(shared)
        want.append(alone)
    _on_threads(workers, 3000)
    for plan, g, w in zip(plans, got, want):
        plan.check_errors()
        assert all(torch.equal(g[n].view(torch.uint8), w[n].view(torch.uint8)) for n in w)


@pytest.mark.parametrize("kind", ["e4m3", "e4m3_block"])
def test_prefills_of_two_topk_at_once(cuda_dev, kind):
    workers, got, want, plans = [], [], [], []
    for topk in (2, 600):
        case = synth.Case("topk", [2000], [2000], 16, 2, 128, 2, 64, topk, kv_dtype=kind)
        inp = synth.make_inputs(case, device=cuda_dev)
        plans.append(make_plan(case, inp))
        idx = torch.from_numpy(random_idx(case, np.random.default_rng(1))).to(cuda_dev)

        def attend(stream=None, plan=plans[-1], inp=inp, idx=idx, **out):
            return plan.sparse_attn(inp["q"], inp["k_pages"], inp["v_pages"], inp["kv_indices"], idx,
                                    k_scale=inp["k_scale"], v_scale=inp["v_scale"], stream=stream, **out)
        want.append(attend())
        got.append(tuple(torch.empty_like(t) for t in want[-1]))
        workers.append(lambda s, attend=attend, o=got[-1]: attend(s, out=o[0], lse=o[1]))
    _on_threads(workers, 3000)
    for plan, g, w in zip(plans, got, want):
        plan.check_errors()
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
