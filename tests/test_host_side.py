"""libmsa's host side over a CUDA runtime of host functions (fake_cudart.cpp):
what it asks of the runtime, and what it leaves behind when memory runs out.
Each test runs a child process that has the fake preloaded."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(ROOT, "block_sparse_long_proxy_gb300", "libmsa.so")

# what every child starts with: the library by its C ABI, and the fake's own calls
PRELUDE = """
import ctypes as C
fake, lib = C.CDLL(%(fake)r), C.CDLL(%(lib)r)
P, I, L = C.c_void_p, C.c_int32, C.c_int64
BF16, E4M3, BLOCK = 0, 1, 2
fake.fake_live_host.restype = fake.fake_live_device.restype = fake.fake_events.restype = C.c_long
fake.fake_fail.argtypes = [C.c_long, C.c_long]
lib.msa_last_error.restype = C.c_char_p
lib.msa_plan.argtypes = [P, P] + [I] * 8 + [L, I, C.c_uint32, P, P]
lib.msa_plan_destroy.argtypes = [P]
lib.msa_kv_append.argtypes = [P, P, P, P, L, P, L] + [P] * 6
lib.msa_pk_append.argtypes = [P, P, P, P, L] + [P] * 8
lib.msa_append_bwd.argtypes = [P] * 12
lib.msa_proxy_maxscore.argtypes = [P] * 6
lib.msa_proxy_maxscore_fp8.argtypes = lib.msa_proxy_topk.argtypes = [P] * 7
lib.msa_proxy_maxscore_nvfp4.argtypes = [P] * 8
lib.msa_sparse_attn.argtypes = [P] * 11
lib.msa_sparse_attn_bwd.argtypes = [P] * 11 + [C.c_float] + [P] * 6

def plan(qo, kv, hq, hkv, d, topk, kind, pages=64):
    n, h = len(qo), P()
    s = lib.msa_plan((I * n)(*qo), (I * n)(*kv), n, hq, hkv, hkv, d, 64, 128, topk, pages, kind, 0, None, C.byref(h))
    return s, h

class Event(C.Structure):
    _fields_ = [("func", P), ("kind", C.c_int), ("bytes", C.c_long)]

def events():
    e = (Event * 4096)()
    return [(x.func, x.kind, x.bytes) for x in e[:fake.fake_events(e, 4096)]]
"""


@pytest.fixture(scope="module")
def child(tmp_path_factory):
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    fake = str(tmp_path_factory.mktemp("fake") / "fake_cudart.so")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(cuda, "include"),
                    os.path.join(HERE, "fake_cudart.cpp"), "-o", fake], check=True)

    def run(body):
        r = subprocess.run([sys.executable, "-c", PRELUDE % dict(fake=fake, lib=LIB) + body], capture_output=True,
                           text=True, timeout=300, env=dict(os.environ, LD_PRELOAD=fake))
        assert r.returncode == 0, (r.returncode, r.stdout[-2000:], r.stderr[-4000:])
        return r.stdout
    return run


def test_one_shared_memory_limit_a_kernel(child):
    """A kernel's limit of dynamic shared memory belongs to the function, for all
    threads of the process: whatever the plan, a kernel is given the same one, so
    that no call lowers it between another's setting and its launch."""
    child("""
at = [P((i + 1) << 20) for i in range(12)]
for kind in (BF16, E4M3, BLOCK):
    for d in (64, 128):
        sc = at[8:10] if kind != BF16 else [None, None]
        for qo, kv in (([1] * 3, [300, 77, 128]), ([300, 5], [300, 700])):
            s, h = plan(qo, kv, 8, 8, d, 4, kind)
            assert s == 0, lib.msa_last_error()
            s = lib.msa_kv_append(h, None, None, at[0], 8 * d, at[1], 8 * d, at[2], at[3], at[4], *sc, None)
            assert s == 0, lib.msa_last_error()
            lib.msa_plan_destroy(h)
        if kind == E4M3 and d == 64:
            continue
        for topk in (1, 16, 200, 1024):
            # whole units, units shared by clusters, rows apart, decode
            for qo, kv in (([9000], [9000]), ([300], [9000]), ([1] * 4 + [2000], [900] * 4 + [9000]), ([1] * 4, [900] * 4)):
                s, h = plan(qo, kv, 16, 2, d, topk, kind, 256)
                assert s == 0, lib.msa_last_error()
                s = lib.msa_sparse_attn(h, at[0], at[1], at[2], at[3], at[4], *sc, at[5], None, None)
                assert s == 0, lib.msa_last_error()
                lib.msa_plan_destroy(h)
limits, launches = {}, 0
for func, kind, n in events():
    if kind == 0:
        limits.setdefault(func, set()).add(n)
    else:
        launches += 1
        assert n <= max(limits.get(func, {0})), (func, n)
assert launches >= 60 and len(limits) >= 12, (launches, len(limits))
apart = {hex(f): sorted(v) for f, v in limits.items() if len(v) > 1}
assert not apart, apart
""")


# plans whose tables differ: prefill and its backward, decode, block scales with tiles of few rows apart
BATCHES = """
BATCHES = [([300, 77, 2000], [300, 1000, 2100], 16, 4, 128, 6, BF16), ([1] * 9, [700 + i for i in range(9)], 16, 4, 128, 6, E4M3),
           ([1] * 30 + [700, 4], [900] * 30 + [1500, 70], 64, 4, 128, 9, BLOCK)]
"""


def test_out_of_host_memory_is_a_status(child):
    """No allocation left from the nth on, whichever that is: msa_plan answers
    MSA_ERR_NO_MEMORY and has a message, which needs no memory either."""
    child(BATCHES + """
for batch in BATCHES:
    for n in range(100000):
        fake.fake_fail(n, -1)
        s, h = plan(*batch)
        fake.fake_fail(-1, -1)
        if s == 0:
            break
        assert s == 4 and not h and lib.msa_last_error() == b"msa_plan: out of host memory", (n, s, lib.msa_last_error())
    assert n > 20
    lib.msa_plan_destroy(h)
""")


def test_a_failed_plan_leaves_nothing_behind(child):
    """Whichever allocation fails, of the host's or the device's, what came before
    it is given back; and so is all of a plan that is destroyed."""
    child(BATCHES + """
left = lambda: (fake.fake_live_host(), fake.fake_live_device())
for batch in BATCHES:
    before = left()
    for n in range(100000):
        fake.fake_fail(n, -1)
        s, h = plan(*batch)
        fake.fake_fail(-1, -1)
        if s == 0:
            break
        assert s == 4 and left() == before, (n, s, before, left())
    assert left()[0] > before[0] and left()[1] == before[1] + 1
    lib.msa_plan_destroy(h)
    assert left() == before
    fake.fake_fail(-1, 0)
    s, h = plan(*batch)
    fake.fake_fail(-1, -1)
    assert s == 4 and left() == before
    for bad in ((batch[0], [0] * len(batch[0])), ([0] * len(batch[0]), batch[1])):
        assert plan(*bad, *batch[2:])[0] == 1 and left() == before
""")


def test_plans_belong_to_their_device(child):
    """Every call of a plan answers MSA_ERR_INVALID_ARG, and launches nothing, while
    another device is current; and works again when the plan's is."""
    child("""
at = [P((i + 1) << 20) for i in range(16)]
def calls(qo, kind):
    s, h = plan(qo, [300] * len(qo), 8, 8, 128, 4, kind)
    assert s == 0
    sc = at[8:10] if kind != BF16 else [None, None]
    yield lambda: lib.msa_kv_append(h, None, None, at[0], 1024, at[1], 1024, at[2], at[3], at[4], *sc, None)
    yield lambda: lib.msa_pk_append(h, None, None, at[0], 64, at[1], at[2], None, None, None, None, None, None)
    yield lambda: lib.msa_proxy_maxscore(h, at[0], at[1], at[2], at[3], None)
    yield lambda: lib.msa_sparse_attn(h, at[0], at[1], at[2], at[3], at[4], *sc, at[5], None, None)
    if max(qo) == 1:
        yield lambda: lib.msa_proxy_maxscore_fp8(h, at[0], at[1], at[2], at[3], at[4], None)
        yield lambda: lib.msa_proxy_maxscore_nvfp4(h, at[0], at[1], at[2], at[3], at[4], at[5], None)
    else:
        yield lambda: lib.msa_proxy_topk(h, at[0], at[1], at[2], None, at[3], None)
    if kind == BF16:
        yield lambda: lib.msa_append_bwd(h, None, None, None, at[0], at[1], None, None, at[2], None, None, None)
        yield lambda: lib.msa_sparse_attn_bwd(h, *at[:10], 1.0, *at[10:15], None)
    lib.msa_plan_destroy(h)
n = 0
for qo in ([1] * 3, [200, 5]):
    for kind in (BF16, E4M3, BLOCK):
        for call in calls(qo, kind):
            before = len(events())
            fake.fake_set_device(1)
            assert call() == 1 and b"belongs to device 0, device 1 is current" in lib.msa_last_error(), lib.msa_last_error()
            assert len(events()) == before
            fake.fake_set_device(0)
            if kind != BF16 or n == 0:
                assert call() == 0, lib.msa_last_error()
                assert len(events()) > before
            n += 1
assert n == 37, n
""")
