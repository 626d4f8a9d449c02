"""The host side of tree and latent attention over a CUDA runtime of host functions:
what is refused, before anything is enqueued, and what a call launches."""
from tests.test_host_side import child  # noqa: F401

CALLS = """
lib.msa_tree_attn.argtypes = [P] * 12
lib.msa_latent_append.argtypes = [P] * 4 + [L, P, L, P, I, I, P, P]
lib.msa_latent_attn.argtypes = [P] * 6 + [I, I, C.c_float, P, P, P]
lib.msa_latent_expand.argtypes = [P] * 5 + [I, I, P, P, P]
lib.msa_rope_create.argtypes = [I, I, C.c_double, I, C.c_double, I, C.c_double, C.c_double, P]
at = [(i + 1) << 20 for i in range(16)]

def tree(h, kind, **kw):
    a = dict(q=at[0], k=at[1], v=at[2], table=at[3], idx=at[4], mask=at[5], ks=at[6] if kind != BF16 else None,
             vs=at[7] if kind != BF16 else None, out=at[8], lse=at[9]) | kw
    return lib.msa_tree_attn(h, *[P(x) if x else None for x in a.values()], None)
def append(h, **kw):
    a = dict(rope=None, pos=None, c=at[0], cs=256, key=at[1], ks=32, table=at[2], n=256, w=32, pages=at[3]) | kw
    p = lambda x: P(x) if x else None
    return lib.msa_latent_append(h, a["rope"], p(a["pos"]), p(a["c"]), a["cs"], p(a["key"]), a["ks"], p(a["table"]), a["n"],
                                 a["w"], p(a["pages"]), None)
def attn(h, **kw):
    a = dict(q=at[0], pages=at[1], table=at[2], idx=at[3], mask=None, n=256, w=32, scale=0.1, out=at[4], lse=None) | kw
    p = lambda x: P(x) if x else None
    return lib.msa_latent_attn(h, p(a["q"]), p(a["pages"]), p(a["table"]), p(a["idx"]), p(a["mask"]), a["n"], a["w"], a["scale"],
                               p(a["out"]), p(a["lse"]), None)
def expand(h, **kw):
    a = dict(pages=at[0], wk=at[1], wv=at[2], table=at[3], n=256, w=32, k=at[4], v=at[5]) | kw
    p = lambda x: P(x) if x else None
    return lib.msa_latent_expand(h, p(a["pages"]), p(a["wk"]), p(a["wv"]), p(a["table"]), a["n"], a["w"], p(a["k"]), p(a["v"]), None)
def launches():
    return sum(kind == 1 for _, kind, _ in events())
def refused(status, call):
    before = launches()
    assert call() == status, (call(), lib.msa_last_error())
    assert launches() == before
"""


def test_refusals(child):  # noqa: F811
    child(CALLS + """
for kind in (BF16, E4M3, BLOCK):
    s, h = plan([5, 128], [300, 128], 8, 2, 128, 4, kind)
    assert s == 0 and tree(h, kind) == 0 and launches() > 0
    for name in ("q", "k", "v", "table", "idx", "mask", "out"):
        refused(1, lambda: tree(h, kind, **{name: None}))
    for name in ("q", "k", "v", "out"):
        refused(1, lambda: tree(h, kind, **{name: at[0] + 8}))
    refused(1, lambda: tree(h, kind, mask=at[5] + 2))
    assert tree(h, kind, mask=at[5] + 4) == 0 and tree(h, kind, lse=None) == 0
    for name in ("ks", "vs"):
        refused(1, lambda: tree(h, kind, **{name: None if kind != BF16 else at[6]}))
    refused(1, lambda: tree(None, kind))
    lib.msa_plan_destroy(h)
s, h = plan([129], [300], 8, 2, 128, 4, BF16)
refused(2, lambda: tree(h, BF16))
refused(2, lambda: attn(h, mask=at[5]))
assert attn(h) == 0
lib.msa_plan_destroy(h)

s, h = plan([5, 1], [300, 1], 8, 2, 128, 4, BF16)
rope = P()
assert lib.msa_rope_create(48, 0, 1e4, 0, 1.0, 0, 0.0, 0.0, C.byref(rope)) == 0
for call, need in ((append, ("c", "key", "table", "pages")), (attn, ("q", "pages", "table", "idx", "out")),
                   (expand, ("pages", "wk", "wv", "table", "k", "v"))):
    assert call(h) == 0
    refused(1, lambda: call(None))
    for name in need:
        refused(1, lambda: call(h, **{name: None}))
        if name not in ("table", "idx"):
            refused(1, lambda: call(h, **{name: at[10] + 8}))
    for n, w in ((0, 32), (64, 32), (320, 32), (640, 32), (-128, 32), (256, 0), (256, 8), (256, 80), (256, -16)):
        refused(2, lambda: call(h, n=n, w=w, **(dict(cs=1024, ks=128) if call is append else {})))
for kw in (dict(cs=248), dict(ks=24), dict(cs=260), dict(rope=rope), dict(ks=1 << 41)):
    refused(1, lambda: append(h, **kw))
assert append(h, cs=288, ks=288) == 0
refused(1, lambda: expand(h, k=at[5]))
refused(1, lambda: expand(h, v=at[5] + 16))
for scale in (0.0, -1.0, float("nan"), float("inf")):
    refused(1, lambda: attn(h, scale=scale))
lib.msa_plan_destroy(h)
s, h = plan([5], [300], 8, 2, 64, 4, BF16)
refused(1, lambda: expand(h, w=64))
lib.msa_plan_destroy(h)
s, h = plan([5], [300], 8, 2, 128, 4, BLOCK)
refused(2, lambda: expand(h))
assert append(h) == 0 and attn(h) == 0
""")


def test_pools_beyond_32_bit_rows(child):  # noqa: F811
    """K/V rows (page, head, slot) are 32-bit coordinates of the tree's loads: a pool of more is
    refused, whatever its type.  A latent cache has one head."""
    child(CALLS + """
for kind in (BF16, E4M3):
    for heads, pages, status in ((8, 1 << 21, 0), (8, (1 << 21) + 1, 1), (1, 1 << 24, 0), (3, 5592405, 0), (3, 5592406, 1)):
        s, h = plan([5], [300], 24, heads, 64, 4, kind, pages)
        assert s == 0
        if status:
            refused(status, lambda: tree(h, kind))
            assert b"2^24" in lib.msa_last_error()
        else:
            assert tree(h, kind) == 0
        assert attn(h) == 0 and append(h) == 0 and (kind != BF16 or expand(h) == 0)
        lib.msa_plan_destroy(h)
""")


def test_plans_belong_to_their_device(child):  # noqa: F811
    child(CALLS + """
s, h = plan([5, 1], [300, 1], 8, 2, 128, 4, BF16)
for call in (lambda: tree(h, BF16), lambda: append(h), lambda: attn(h), lambda: expand(h)):
    fake.fake_set_device(1)
    refused(1, call)
    assert b"belongs to device 0, device 1 is current" in lib.msa_last_error()
    fake.fake_set_device(0)
    assert call() == 0
""")


def test_one_limit_of_shared_memory_a_kernel(child):  # noqa: F811
    """Plans of any topk ask for one limit, and launch within it."""
    child(CALLS + """
limit = {}
for topk in (1, 16, 1024):
    for qo in ([1], [3], [8, 1], [3, 60], [128]):
        for kind in (BF16, E4M3, BLOCK):
            s, h = plan(qo, [300] * len(qo), 16, 2, 128, topk, kind)
            assert s == 0 and tree(h, kind) == 0 and attn(h) == 0
            lib.msa_plan_destroy(h)
for func, kind, size in events():
    if kind == 0:
        assert limit.setdefault(func, size) == size
    else:
        assert size <= limit[func] <= 232448, (size, limit[func])
assert len(limit) >= 3, len(limit)
""")


def test_wide_trees_take_the_rows(child):  # noqa: F811
    """The batches of wide trees that the GPU tests run all go through one kernel, and
    narrow ones through others."""
    import json
    from tests.test_tree_attn_gpu import SHAPES, WIDE
    child(CALLS + "import json\nSHAPES, WIDE = (json.loads(x) for x in %r)" % ([json.dumps(list(x.values())) for x in (SHAPES, WIDE)],) + """
def kernel(qo, kv, hq, hkv, hp, topk, d, kind):
    n, h = len(qo), P()
    assert lib.msa_plan((I * n)(*qo), (I * n)(*kv), n, hq, hkv, hp, d, 64, 128, topk, 4096, kind, 0, None, C.byref(h)) == 0
    before = len(events())
    assert tree(h, kind) == 0
    lib.msa_plan_destroy(h)
    return [f for f, k, _ in events()[before:] if k == 1]
for d in (64, 128):
    for kind in (BF16, E4M3, BLOCK):
        narrow = {f for s in SHAPES for f in kernel(*s, d, kind)}
        wide = {f for s in WIDE for f in kernel(*s, d, kind)}
        assert len(wide) == 1 and len(narrow - wide) > 1, (d, kind, wide, narrow)
""")


def test_the_next_launch_starts_behind_the_tensor_memory():
    """A CTA that lets the next launch start has its tensor memory: one of that launch could
    otherwise take what it still waits for, and then wait for it to end."""
    import os
    import re
    from tests.test_host_side import ROOT
    for name, kernels in (("columns.cu", 2), ("expand.cu", 1)):
        with open(os.path.join(ROOT, "block_sparse_long_proxy_gb300", "csrc", name)) as f:
            bodies = re.split(r"__global__", f.read())[1:]
        assert len(bodies) == kernels
        for body in bodies:
            alloc = re.search(r"tmem_alloc\(|tcgen05\.alloc", body).start()
            there = body.index("__syncthreads();", alloc)
            assert body.count("pdl_trigger();") == 1 and body.index("pdl_trigger();") > there


def test_nothing_is_under_way_when_a_cta_leaves():
    """After a wait that was given up, too, a CTA waits (bounded) for its loads and products before
    it frees its tensor memory: the producers for what they issued last, the issuer for a commit
    behind all of its products."""
    import os
    import re
    from tests.test_host_side import ROOT
    for name, kernels in (("columns.cu", 2), ("expand.cu", 1)):
        with open(os.path.join(ROOT, "block_sparse_long_proxy_gb300", "csrc", name)) as f:
            bodies = re.split(r"__global__", f.read())[1:]
        assert len(bodies) == kernels
        for body in bodies:
            commit = re.search(r"(mma_commit_if\(leader, |commit_pair\()drain", body).start()
            waits = [m.start() for m in re.finditer(r"(?<!= )(?<!\()mbar_wait_inl\((a_|b_|tail_)?full \+ [^;]*a\.err\);", body)]
            products = [m.start() for m in re.finditer(r"\bmma_(ss_if|ts_if|pair)\(leader", body)]
            free = max(m.start() for m in re.finditer(r"tmem_dealloc\(|tcgen05\.dealloc", body))
            assert max(products) < commit < body.index("drain, 0", commit) < free
            assert len(waits) == (2 if "tail_full" in body or name == "expand.cu" else 1) and max(waits) < free
