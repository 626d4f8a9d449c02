"""What libmsa uploads and launches, over a CUDA runtime of host functions that counts
both (fake_launches.cpp)."""
import os
import shutil
import subprocess
import sys

import pytest

from tests.test_host_side import HERE, LIB, PRELUDE, ROOT

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
                           text=True, timeout=600, cwd=ROOT, env=dict(os.environ, LD_PRELOAD=fake))
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


# kernels by name: the symbols of the host's side of a launch
NAMES = """
import re, subprocess
from tests.test_tree_latent_host import CALLS
exec(CALLS)
fake.fake_last_func.restype = P
at0 = C.cast(lib.msa_version, P).value
NAMES = {}
for line in subprocess.run(["nm", "-C", lib._name], capture_output=True, text=True, check=True,
                           env={k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}).stdout.splitlines():
    m = re.match(r"([0-9a-f]+) [tT] (.*)", line)
    if m and "[clone" not in m[2] and "__device_stub__" not in m[2]:
        # (an enumerator may be printed with its type before it)
        n = re.sub(r"\\(anonymous namespace\\)::|msa::|^void |\\(Cache\\)", "", m[2])
        NAMES[n.split("(")[0]] = int(m[1], 16)
at0 -= NAMES["msa_version"]
BY_PLACE = {a: n for n, a in NAMES.items()}
OURS = {n for n in NAMES if re.match(r"(columns|rows|expand)_kernel<", n)}
def launched():
    return BY_PLACE[fake.fake_last_func() - at0], fake.fake_last_cluster()
def plan_of(qo, kv, hq, hkv, hp, d, topk, kind):
    n, h = len(qo), P()
    s = lib.msa_plan((I * n)(*qo), (I * n)(*kv), n, hq, hkv, hp, d, 64, 128, topk, 1 << 16, kind, 0, None, C.byref(h))
    assert s == 0, lib.msa_last_error()
    return h
"""


def test_every_instance_is_tested(child):
    """Each kernel of tree and latent attention and of the expansion is what some batch of the
    GPU tests is given, the batches of tree_instances.py the one that they stand for: an
    estimate measured anew that drops one shows here."""
    if shutil.which("nm") is None:
        pytest.skip("no nm")
    child("import os\n" + NAMES + """
from tests.tree_instances import LATENTS, TREES, batch, boxed
got = set()
for kinds, table in (((BF16,), TREES["bf16"]), ((E4M3, BLOCK), TREES["fp8"])):
    for (cols, two, parts, d, box), (n, rows, ctx, hq, hkv, hp, topk) in table:
        for kind in kinds:
            h = plan_of(*batch(n, rows, ctx), hq, hkv, hp, d, topk, kind)
            assert tree(h, kind) == 0
            name = ("columns_kernel<%d, %d, %s>" % (kind != BF16, cols, "true" if two else "false") if cols else
                    "rows_kernel<%s, %d>" % ("true" if kind else "false", d))
            assert launched() == (name, parts), (launched(), name, parts, n, rows, ctx, hq, hkv, hp, topk)
            assert box is None or box == boxed(cols, hq, hp)
            got.add(name)
            lib.msa_plan_destroy(h)
for (cols, parts, latent, box), (n, rows, ctx, hq, hkv, hp, topk) in LATENTS:
    h = plan_of(*batch(n, rows, ctx), hq, hkv, hp, 128, topk, BF16)
    assert attn(h, n=latent) == 0
    name = "columns_kernel<2, %d, false>" % cols
    assert launched() == (name, parts) and box == boxed(cols, hq, hp)
    got.add(name)
    lib.msa_plan_destroy(h)
h = plan_of([512, 77], [3000, 900], 32, 1, 1, 128, 9, BF16)      # test_latent_chunk
for latent in (512, 384, 256, 128):
    assert attn(h, n=latent, w=64) == 0 and launched() == ("columns_kernel<2, 64, false>", 1)
for d, rope in ((64, 16), (64, 32), (64, 48), (128, 16), (128, 32), (128, 48), (128, 64)):  # test_expand_of_every_width
    h = plan_of([1] * 3, [300, 5, 128], 7, 7, 7, d, 1, BF16)
    assert expand(h, w=rope) == 0
    got.add(launched()[0])
assert len(OURS) == 25 and got == OURS, (sorted(OURS - got), sorted(got - OURS))
""")
