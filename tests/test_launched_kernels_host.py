"""What libmsa uploads and launches, over a CUDA runtime of host functions that counts
both (fake_launches.cpp)."""
import os
import subprocess
import sys

import pytest

from tests.test_host_side import HERE, LIB, PRELUDE

COUNTS = """
fake.fake_uploaded.restype = C.c_long
def uploaded(*a, **kw):
    before = fake.fake_uploaded()
    s, h = plan(*a, **kw)
    assert s == 0, lib.msa_last_error()
    lib.msa_plan_destroy(h)
    return fake.fake_uploaded() - before
"""


@pytest.fixture(scope="module")
def child(tmp_path_factory):
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    fake = str(tmp_path_factory.mktemp("fake") / "fake_launches.so")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(cuda, "include"),
                    os.path.join(HERE, "fake_launches.cpp"), "-o", fake], check=True)

    def run(body):
        r = subprocess.run([sys.executable, "-c", PRELUDE % dict(fake=fake, lib=LIB) + COUNTS + body], capture_output=True,
                           text=True, timeout=600, env=dict(os.environ, LD_PRELOAD=fake))
        assert r.returncode == 0, (r.returncode, r.stdout[-2000:], r.stderr[-4000:])
        return r.stdout
    return run


def test_a_plan_uploads_a_byte_a_page_table_entry(child):
    """What the expansion of a latent cache needs of every page, for all plans of bf16: it is
    made and uploaded with each plan, of long contexts too (32 x 131072 keys: 32768 entries)."""
    child("""
for qo, kv in (([8] * 32, [131072] * 32), ([1] * 32, [131071] * 32), ([5, 1], [1 << 20, 300])):
    entries = sum((k + 127) // 128 for k in kv)
    of = {kind: uploaded(qo, kv, 64, 8, 128, 16, kind, 1 << 16) for kind in (BF16, E4M3)}
    few = {kind: uploaded(qo, [max(q, 8) for q in qo], 64, 8, 128, 16, kind, 1 << 16) for kind in (BF16, E4M3)}
    # tables by blocks of keys are alike in both kinds, but for 256-byte borders
    assert (of[BF16] - few[BF16]) - (of[E4M3] - few[E4M3]) <= entries + 1024, (entries, of, few)
""")
