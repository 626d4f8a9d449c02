"""The cache-side operators of libmsa as cases to measure: rotary positions, the
paged-cache append with its quantisers and its backward, and block-sparse
attention over a cache held in e4m3 with one scale for each (page, KV head).

Each operator has a plain form in elementary torch operations (fp32, angles
in fp64) and the library's call; `own` says which of the two run() takes.
"""
import math
import random

import torch

own = False

PAGE = 128
E_MIN, E_MAX = -40, 40          # exponents of a block scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases --

def listed():
    def rope(name, rows, heads, **kw):
        return dict(name=name, op="rope", rows=rows, heads=heads, d=128, rot=128, layout="half", scaling="none",
                    factor=1.0, dtype="bf16", inverse=False, gap=0, first=0) | kw

    def cache(name, op, **kw):
        return dict(name=name, op=op, batch=1, rows=1, ctx=0, even=True, lens=0, hkv=8, d=128, dp=64, kv="e4m3_block",
                    rot=128, layout="half", scaling="none", factor=1.0) | kw

    def attn(name, **kw):
        return dict(name=name, op="attn", batch=1, rows=1, ctx=0, even=True, lens=0, hq=64, hkv=8, hp=8, topk=16) | kw

    return [
        # one decode step of 32 sequences: the new tokens' queries, at far positions (latency)
        rope("rotate q decode", 32, 64, first=131000),
        # the queries of a 32K prefill, taken out of a q|k|v projection; interleaved pairs, half the head rotated,
        # positions scaled to a longer context
        rope("rotate q prefill 32K", 32768, 32, layout="interleaved", rot=64, scaling="yarn", factor=4.0, gap=2048),
        # the attention's fp32 dq of a 64K training step, rotated back
        rope("rotate dq back 64K", 65536, 32, dtype="fp32", inverse=True),
        # one decode step of 32 sequences: a token's K and V into pages that are partly filled (latency)
        cache("append K V decode", "kv", batch=32, ctx=2000, even=False, lens=3),
        # the K and V of a 32K prefill into an empty cache
        cache("append K V prefill 32K", "kv", rows=32768),
        # the proxy keys of ragged chunks, kept in bf16 for the prefill and in NVFP4 for the decode steps after it
        cache("append proxy K chunks", "pk", batch=5, rows=7000, ctx=5000, even=False, lens=5, rot=32),
        # the gradient pages of a 64K training step back to rows, with the rotation's transpose
        cache("append backward 64K", "bwd", rows=65536),
        # a single user's decode step at 131072 keys
        attn("attend decode 1", ctx=131071),
        # a serving batch's decode step
        attn("attend decode 32", batch=32, ctx=32767),
        # a small ragged decode batch, sixteen query heads a KV head
        attn("attend decode ragged", batch=7, ctx=5000, even=False, lens=11, hq=32, hkv=2, hp=2, topk=5),
        # chunks of a mixed batch on top of what their sequences hold already; three query heads a KV head
        attn("attend chunks ragged", batch=6, rows=700, ctx=9000, even=False, lens=13, hq=12, hkv=4, hp=4, topk=9),
        # the 32K prefill
        attn("attend prefill 32K", rows=32768, hq=32),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "kv", "pk", "bwd", "attn", "attn"])
    layout = rng.choice(["half", "interleaved"])
    scaling = rng.choice(["none", "linear", "ntk", "yarn"])
    factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0])
    if op == "rope":
        d = rng.choice([32, 64, 128])
        heads = rng.randint(1, 64)
        return dict(op=op, rows=_log_int(rng, 1, 65536 * 32 // heads if heads > 32 else 65536), heads=heads, d=d,
                    rot=16 * rng.randint(1, d // 16), layout=layout, scaling=scaling, factor=factor,
                    dtype=rng.choice(["bf16", "fp32"]), inverse=rng.random() < 0.5, gap=8 * rng.randint(0, 200),
                    first=_log_int(rng, 1, 1000000))
    batch = _log_int(rng, 1, 40)
    if op in ("kv", "pk", "bwd"):
        d, dp = rng.choice([64, 128]), rng.choice([32, 64])
        width = dp if op == "pk" else min(d, dp) if op == "bwd" else d
        return dict(op=op, batch=batch, rows=_log_int(rng, 1, 32768 // batch), ctx=_log_int(rng, 1, 32768 // batch),
                    even=False, lens=rng.randint(0, 10**6), hkv=rng.randint(1, 8), d=d, dp=dp,
                    kv=rng.choice(["bf16", "e4m3", "e4m3_block"]), rot=16 * rng.randint(1, width // 16), layout=layout,
                    scaling=scaling, factor=factor)
    hkv, m = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2])
    group = rng.choice([1, 3, 4, 8, 16 // m])
    decode = rng.random() < 0.5
    return dict(op=op, batch=batch, rows=1 if decode else _log_int(rng, 2, 4096 // batch),
                ctx=_log_int(rng, 1, 200000 // batch), even=False, lens=rng.randint(0, 10**6), hq=hkv * m * group,
                hkv=hkv, hp=hkv * m, topk=_log_int(rng, 1, 24))


def _lens(case):
    """(qo_lens, kv_lens): new rows and keys of each sequence."""
    if case["even"]:
        return [case["rows"]] * case["batch"], [case["rows"] + case["ctx"]] * case["batch"]
    r = random.Random(case["lens"])
    qo = [r.randint(1, case["rows"]) for _ in range(case["batch"])]
    return qo, [q + r.randint(0, case["ctx"]) for q in qo]


def _blocks(n):
    return (n + PAGE - 1) // PAGE


def work(case):
    if case["op"] == "rope":
        n = case["rows"] * case["heads"] * case["d"]
        return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4) + 4 * case["rows"], "flops": 3 * n}
    qo, kv = _lens(case)
    rows = sum(qo)
    pages = sum(_blocks(k) - (k - q) // PAGE for q, k in zip(qo, kv))        # pages that get a row
    if case["op"] == "kv":
        n = 2 * rows * case["hkv"] * case["d"]
        scales = 8 * pages * case["hkv"] if case["kv"] == "e4m3_block" else 0
        return {"bytes": n * (4 if case["kv"] == "bf16" else 3) + scales + 4 * rows, "flops": 4 * n}
    if case["op"] == "pk":
        n = rows * case["dp"]
        return {"bytes": n * 4 + n // 2 + n // 16 + 4 * rows, "flops": 5 * n}
    if case["op"] == "bwd":
        n = rows * (2 * case["hkv"] * case["d"] + case["dp"])
        return {"bytes": 8 * n + 4 * rows, "flops": 2 * n}
    d, total, flops, sel = 128, sum(qo), 0, 0
    for q, k in zip(qo, kv):
        for r0 in range(0, q, PAGE):
            n = min(PAGE, q - r0)
            nb = min(case["topk"], (k - q + r0 + n - 1) // PAGE + 1)
            flops += 4 * d * n * case["hq"] * nb * PAGE
            sel += nb * case["hp"]
    pages = min(sel, sum(_blocks(k) for k in kv) * case["hkv"])
    return {"bytes": total * case["hq"] * (4 * d + 4) + pages * (2 * PAGE * d + 8) + 4 * sel, "flops": flops}


# ------------------------------------------------------------------ inputs --

def _freqs(rot, scaling, factor, base=10000.0, length=4096, beta_fast=32.0, beta_slow=1.0):
    """Turns a position of each pair, and the factor on the rotated values."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    turns = base ** (-2.0 * i / rot) / (2 * math.pi)
    if scaling == "linear":
        turns = turns / factor
    if scaling != "yarn":
        return turns, 1.0
    dim = lambda beta: rot * math.log(length / (2 * math.pi * beta)) / (2 * math.log(base))  # noqa: E731
    lo, hi = math.floor(dim(beta_fast)), math.ceil(dim(beta_slow))
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return turns * (1 - ramp) + turns / factor * ramp, 0.1 * math.log(factor) + 1 if factor > 1 else 1.0


def _rope_of(case):
    from block_sparse_long_proxy_gb300 import msa
    return msa.Rope(case["rot"], layout=case["layout"], scaling=case["scaling"], factor=case["factor"],
                    original_len=4096)


def _block_codes(shape, lo, hi, gen):
    """e4m3 codes of every page, and a power-of-two scale for each (page, head)."""
    x = torch.randn(shape, generator=gen, device="cuda")
    codes = x.mul_(110.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return codes, torch.exp2(torch.randint(lo, hi + 1, shape[:2], generator=gen, device="cuda").float())


def _tables(qo, kv, gen):
    """What a serving program holds on the device beside the cache: the page
    table, and each new row's position and place."""
    nb = [_blocks(k) for k in kv]
    num_pages = sum(nb) + 3
    table = torch.randperm(num_pages, generator=gen, device="cuda")[:sum(nb)].to(torch.int32)
    pos = torch.cat([torch.arange(k - q, k, device="cuda") for q, k in zip(qo, kv)])
    base, entry, first = 0, [], {}
    for q, k, n in zip(qo, kv, nb):
        for j in range((k - q) // PAGE, n):
            first[base + j] = max(0, k - q - j * PAGE)
        entry.append(base + torch.arange(k - q, k, device="cuda") // PAGE)
        base += n
    entry = torch.cat(entry)
    touched = torch.tensor(list(first), device="cuda")
    return dict(num_pages=num_pages, kv_indices=table, positions=pos.to(torch.int32), page=table.long()[entry],
                slot=pos % PAGE, touched=table.long()[touched], first=torch.tensor(list(first.values()), device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 2 + 1)
    if case["op"] == "attn":
        return _prepare_attn(case, gen)
    s = dict(case=case)
    turns, s["mscale"] = _freqs(case["rot"], case["scaling"], case["factor"])
    s["turns"] = turns.cuda()
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    if own:
        s["rope"] = _rope_of(case)
    if case["op"] == "rope":
        t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        wide = rand(case["rows"], case["heads"] * case["d"] + case["gap"]).to(t)
        s["x"] = wide[:, :case["heads"] * case["d"]].unflatten(1, (case["heads"], case["d"]))
        s["out"] = torch.empty(s["x"].shape, dtype=t, device="cuda")
        s["positions"] = torch.arange(case["first"], case["first"] + case["rows"], device="cuda", dtype=torch.int32)
        return s
    qo, kv = _lens(case)
    s |= _tables(qo, kv, gen)
    rows, p, hkv, d, dp = sum(qo), s["num_pages"], case["hkv"], case["d"], case["dp"]
    if own:
        from block_sparse_long_proxy_gb300 import msa
        kind = case["kv"] if case["op"] == "kv" else "bf16"
        s["plan"] = msa.Plan(qo, kv, hkv, hkv, hkv, d, dp, 1, p, kv_dtype=kind)
    if case["op"] == "bwd":
        s |= dict(dk_pages=rand(p, hkv, PAGE, d), dv_pages=rand(p, hkv, PAGE, d), dpk_pages=rand(p, 1, PAGE, dp))
        return s
    if case["op"] == "pk":
        s["pk"] = (rand(rows, 1, dp) * 1.5).to(torch.bfloat16)
        s["pk_pages"] = rand(p, 1, PAGE, dp).to(torch.bfloat16)
        s["codes"] = torch.randint(0, 256, (p, 1, PAGE, dp // 2), generator=gen, device="cuda").to(torch.uint8)
        s["scales"] = (rand(p, 1, PAGE, dp // 16).abs() * 100).clamp(max=448).to(torch.float8_e4m3fn)
        s["global"] = torch.full((1,), 8.0 / (448 * 6), device="cuda")
        s["borders"] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device="cuda")
        pairs = torch.arange(256)
        mags = torch.tensor(E2M1 + tuple(-x for x in E2M1))
        s["values"] = torch.stack([mags[pairs & 15], mags[pairs >> 4]], 1).to(torch.bfloat16).cuda()
        return s
    # K and V as slices of one projection's rows
    wide = rand(rows, 2 * hkv * d).to(torch.bfloat16)
    s["k"], s["v"] = (wide[:, i * hkv * d:(i + 1) * hkv * d].unflatten(1, (hkv, d)) for i in (0, 1))
    if case["kv"] == "bf16":
        s |= dict(k_pages=rand(p, hkv, PAGE, d).to(torch.bfloat16), v_pages=rand(p, hkv, PAGE, d).to(torch.bfloat16),
                  k_scale=None, v_scale=None)
        return s
    s["k_pages"], ks = _block_codes((p, hkv, PAGE, d), -9, -5, gen)
    s["v_pages"], vs = _block_codes((p, hkv, PAGE, d), -9, -5, gen)
    if case["kv"] == "e4m3":        # one scale a head, measured by calibration
        ks, vs = (0.01 * (1 + torch.rand(hkv, generator=gen, device="cuda")) for _ in range(2))
    return s | dict(k_scale=ks, v_scale=vs)


def _prepare_attn(case, gen):
    qo, kv = _lens(case)
    s = dict(case=case) | _tables(qo, kv, gen)
    p, hkv, hp, topk = s["num_pages"], case["hkv"], case["hp"], case["topk"]
    s["q"] = torch.randn((sum(qo), case["hq"], 128), generator=gen, device="cuda").to(torch.bfloat16)
    s["k_pages"], s["k_scale"] = _block_codes((p, hkv, PAGE, 128), -8, -6, gen)
    s["v_pages"], s["v_scale"] = _block_codes((p, hkv, PAGE, 128), -10, -5, gen)
    # what was never written behind a sequence's last key holds any bytes, NaN among them
    last, base = [], 0
    for k in kv:
        base += _blocks(k)
        last.append((base - 1, (k - 1) % PAGE + 1))
    for e, n in last if len(last) < 64 else last[:64]:
        s["k_pages"].view(torch.uint8)[s["kv_indices"][e].long(), :, n:] = 0x7F
        s["v_pages"].view(torch.uint8)[s["kv_indices"][e].long(), :, n:] = 0x7F
    # the tiles of 128 query rows, and a selection for each (tile, proxy head):
    # the diagonal block and other blocks up to it, ascending, padded with -1
    tiles, q0, base = [], 0, 0
    for q, k in zip(qo, kv):
        for r in range(0, q, PAGE):
            n = min(PAGE, q - r)
            tiles.append((q0 + r, n, k - q + r, k, base, (k - q + r + n - 1) // PAGE + 1))
        q0, base = q0 + q, base + _blocks(k)
    s["tiles"] = torch.tensor(tiles, device="cuda")
    s["widest"] = min(PAGE, max(t[1] for t in tiles))
    nvp = s["tiles"][:, 5]
    wide = max(topk, max(t[5] for t in tiles))
    j = torch.arange(wide, device="cuda")
    score = torch.rand((len(tiles), hp, wide), generator=gen, device="cuda")
    score = torch.where(j == nvp[:, None, None] - 1, 2.0, torch.where(j < nvp[:, None, None], score, -1.0))
    top, at = score.topk(topk, dim=-1)
    at = torch.where(top < 0, wide, at).sort(-1).values
    s["idx"] = torch.where(at == wide, -1, at).to(torch.int32).contiguous()
    if own:
        from block_sparse_long_proxy_gb300 import msa
        s["plan"] = msa.Plan(qo, kv, case["hq"], hkv, hp, 128, 64, topk, p, kv_dtype="e4m3_block")
    return s


# --------------------------------------------------------------------- run --

def run(s):
    op = s["case"]["op"]
    if op == "rope":
        if own:
            return s["rope"].apply(s["x"], s["positions"], out=s["out"], inverse=s["case"]["inverse"])
        return _rotate(s, s["x"], s["case"]["inverse"]).to(s["x"].dtype)
    if op == "kv":
        if own:
            s["plan"].kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["kv_indices"], k_scale=s["k_scale"],
                                v_scale=s["v_scale"], rope=s["rope"], positions=s["positions"])
        else:
            _append(s, _rotate(s, s["k"]), s["k_pages"], s["k_scale"])
            _append(s, s["v"].float(), s["v_pages"], s["v_scale"])
        scales = () if s["case"]["kv"] != "e4m3_block" else (s["k_scale"], s["v_scale"])
        return (s["k_pages"], s["v_pages"], *scales)
    if op == "pk":
        if own:
            s["plan"].pk_append(s["pk"], s["kv_indices"], pk_pages=s["pk_pages"], pk_codes=s["codes"],
                                pk_block_scales=s["scales"], pk_global_scale=s["global"], rope=s["rope"],
                                positions=s["positions"])
        else:
            _append_proxy(s)
        return s["pk_pages"], s["values"][s["codes"].int()], s["scales"]
    if op == "bwd":
        if own:
            return s["plan"].append_bwd(s["kv_indices"], dk_pages=s["dk_pages"], dv_pages=s["dv_pages"],
                                        dpk_pages=s["dpk_pages"], k_rope=s["rope"], positions=s["positions"])
        take = lambda pages: pages[s["page"], :, s["slot"]]  # noqa: E731
        return _rotate(s, take(s["dk_pages"]), True), take(s["dv_pages"]), take(s["dpk_pages"])
    if own:
        return s["plan"].sparse_attn(s["q"], s["k_pages"], s["v_pages"], s["kv_indices"], s["idx"],
                                     k_scale=s["k_scale"], v_scale=s["v_scale"])
    return _attend(s)


def _rotate(s, x, inverse=False):
    """x [rows, heads, d] rotated in fp32, by angles taken in fp64."""
    rot, half = s["case"]["rot"], s["case"]["layout"] == "half"
    turns = s["positions"].double()[:, None] * s["turns"]
    angle = (turns - torch.floor(turns)) * (2 * math.pi)
    c, sn = (angle.cos() * s["mscale"]).float()[:, None], (angle.sin() * s["mscale"]).float()[:, None]
    if inverse:
        sn = -sn
    x = x.float()
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if half else (x[..., 0:rot:2], x[..., 1:rot:2])
    y = (a * c - b * sn, b * c + a * sn)
    y = torch.cat(y, -1) if half else torch.stack(y, -1).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _block_scale(amax):
    """The least power of two s with amax <= 448 s, its exponent in [-40, 40]."""
    m, e = torch.frexp(amax.double() / 448)
    e = torch.where(amax > 0, torch.where(m == 0.5, e - 1, e), E_MIN).clamp(E_MIN, E_MAX)
    return torch.exp2(e.float())


def _append(s, x, pages, scale):
    """Rows x [rows, heads, d] in fp32 to their pages and slots."""
    kind, page, slot = s["case"]["kv"], s["page"], s["slot"]
    heads = torch.arange(x.shape[1], device=x.device)
    at = (page[:, None], heads, slot[:, None])
    if kind == "bf16":
        pages[at] = x.to(torch.bfloat16)
        return
    raw = pages.view(torch.uint8)
    if kind == "e4m3_block":
        t, first = s["touched"], s["first"]
        amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")[t]
        before = torch.where(first[:, None] > 0, scale[t], 0.0)
        after = torch.maximum(before, _block_scale(amax))
        moved = (pages[t].float() * (before / after)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        kept = torch.arange(PAGE, device=x.device)[None] < first[:, None]
        raw[t] = torch.where(kept[:, None, :, None], moved, raw[t])
        scale[t] = after
        by = scale[page]
    else:
        by = scale[None]
    raw[at] = (x / by[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _nearest(a, borders):
    """The code of each a >= 0, of codes with these borders between them; on a border the even one."""
    up, down = torch.bucketize(a, borders, right=True), torch.bucketize(a, borders)
    return torch.where(up % 2 == 0, up, down)


def _append_proxy(s):
    x = _rotate(s, s["pk"])[:, 0]
    page, slot = s["page"], s["slot"]
    s["pk_pages"][page, 0, slot] = x.to(torch.bfloat16)
    # both roundings in fp64: bf16 keys over a scale meet the borders between codes
    g, x = s["global"].double(), x.double().unflatten(-1, (-1, 16))
    e4m3 = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    bs = _nearest(x.abs().amax(-1) / (6 * g), (e4m3[1:] + e4m3[:-1]) / 2).to(torch.uint8).view(torch.float8_e4m3fn)
    by = bs.double()[..., None] * g
    y = torch.where(by > 0, x / by, 0.0)
    code = _nearest(y.abs(), s["borders"]) + torch.where(torch.signbit(y), 8, 0)
    code = code.flatten(1).to(torch.uint8)
    s["codes"][page, 0, slot] = code[:, 0::2] | (code[:, 1::2] << 4)
    s["scales"].view(torch.uint8)[page, 0, slot] = bs.view(torch.uint8)


def _attend(s):
    """Every (tile, proxy head) at once: its rows against its gathered blocks."""
    q, idx, tiles, d = s["q"], s["idx"].long(), s["tiles"], 128
    nt, hp, topk = idx.shape
    hq, g = q.shape[1], q.shape[1] // hp
    head = torch.arange(hp, device=q.device) // (hp // s["case"]["hkv"])
    page = s["kv_indices"].long()[tiles[:, 4, None, None] + idx.clamp(min=0)]
    at = (page, head[None, :, None])
    k, v = (s[n].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() for n in ("k_pages", "v_pages"))
    ks, vs = s["k_scale"][at], s["v_scale"][at]
    key = idx[..., None] * PAGE + torch.arange(PAGE, device=q.device)
    there = (idx[..., None] >= 0) & (key < tiles[:, 3, None, None, None])
    v = torch.where(there[..., None], v * vs[..., None, None], 0.0).reshape(nt * hp, topk * PAGE, d)
    k = (k * ks[..., None, None]).reshape(nt * hp, topk * PAGE, d)
    r = torch.arange(s["widest"], device=q.device)
    row = (tiles[:, 0, None] + r).clamp(max=q.shape[0] - 1)
    x = q.float()[row].unflatten(2, (hp, g)).permute(0, 2, 3, 1, 4).reshape(nt * hp, -1, d)
    sc = torch.bmm(x, k.transpose(1, 2)).reshape(nt, hp, g, len(r), -1) / math.sqrt(d)
    pos = tiles[:, 2, None] + r
    seen = (there.reshape(nt, hp, 1, -1) & (key.reshape(nt, hp, 1, -1) <= pos[:, None, :, None]))[:, :, None]
    sc = torch.where(seen, sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    o = torch.bmm(e.reshape(nt * hp, -1, topk * PAGE), v).reshape(nt, hp, g, len(r), d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + torch.log(total))[..., 0]
    good = r < tiles[:, 1, None]
    rows = row[good]
    out, out_lse = torch.empty_like(q), torch.empty(q.shape[:2], device=q.device)
    out[rows] = o.permute(0, 3, 1, 2, 4).reshape(nt, len(r), hq, d)[good].to(torch.bfloat16)
    out_lse[rows] = lse.permute(0, 3, 1, 2).reshape(nt, len(r), hq)[good]
    return out, out_lse


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    """run()'s outputs from the definitions, in fp64."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _turned(s, s["x"], case["inverse"])
    if op == "bwd":
        rows = [t[s["page"], :, s["slot"]].double() for t in (s["dk_pages"], s["dv_pages"], s["dpk_pages"])]
        return _turned(s, rows[0], True), rows[1], rows[2]
    if op == "kv":
        pages, scales = [], []
        for x, p, sc in ((_turned(s, s["k"]), s["k_pages"], s["k_scale"]),
                         (s["v"].double(), s["v_pages"], s["v_scale"])):
            p = p.double()
            h = torch.arange(x.shape[1], device=x.device)
            if case["kv"] == "bf16":
                p[s["page"][:, None], h, s["slot"][:, None]] = x
            elif case["kv"] == "e4m3":
                p[s["page"][:, None], h, s["slot"][:, None]] = _to_e4m3(x / sc.double()[None, :, None])
            else:
                sc = sc.double()
                for t, f in zip(s["touched"].tolist(), s["first"].tolist()):
                    mine = s["page"] == t
                    y, slots = x[mine], s["slot"][mine]
                    a = y.abs().amax((0, 2))
                    e = torch.ceil(torch.log2(a / 448))
                    e = torch.where(a <= 448 * 2.0 ** (e - 1), e - 1, torch.where(a > 448 * 2.0 ** e, e + 1, e))
                    new = 2.0 ** torch.where(a > 0, e, -40.0).clamp(-40, 40)
                    one = p[t]
                    if f:
                        new = torch.maximum(new, sc[t])
                        one[:, :f] = _to_e4m3(one[:, :f] * (sc[t] / new)[:, None, None])
                    one[:, slots] = _to_e4m3(y / new[:, None]).transpose(0, 1)
                    sc[t] = new
                scales.append(sc)
            pages.append(p)
        return (*pages, *scales)
    if op == "pk":
        x = _turned(s, s["pk"])
        pages, fours, bss = s["pk_pages"].double(), s["values"][s["codes"].long()].double(), s["scales"].double()
        pages[s["page"], 0, s["slot"]] = x[:, 0]
        g = s["global"].double()
        blocks = x.reshape(len(x), -1, 16)
        bs = _to_e4m3(blocks.abs().amax(-1) / (6 * g))
        y = blocks / (bs * g).clamp(min=1e-300)[..., None]
        mags = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
        # nearest of the eight; of two equally near, the one with the even code
        dist = (y.abs()[..., None] - mags).abs() + torch.tensor([0, 1e-13] * 4, dtype=torch.float64, device=x.device)
        val = mags[dist.argmin(-1)] * torch.where(torch.signbit(y), -1.0, 1.0)
        fours[s["page"], 0, s["slot"]] = torch.where(bs[..., None] > 0, val, 0.0).reshape(len(x), -1, 2)
        bss[s["page"], 0, s["slot"]] = bs
        return pages, fours, bss
    # attention: one tile after the other
    q, d = s["q"].double(), 128
    o, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    hp, hkv = case["hp"], case["hkv"]
    g = case["hq"] // hp
    for (q0, n, pos0, kv_len, base, _), sel in zip(s["tiles"].tolist(), s["idx"].tolist()):
        for p in range(hp):
            blocks = [j for j in sel[p] if j >= 0]
            if not blocks:
                continue
            at = s["kv_indices"].long()[torch.tensor(blocks, device=q.device) + base]
            h = p // (hp // hkv)
            keys = torch.cat([torch.arange(j * PAGE, (j + 1) * PAGE) for j in blocks]).to(q.device)
            k, v = ((s[a].view(torch.uint8)[at, h].view(torch.float8_e4m3fn).double()
                     * s[b][at, h].double()[:, None, None]).flatten(0, 1)
                    for a, b in (("k_pages", "k_scale"), ("v_pages", "v_scale")))
            k, v, keys = k[keys < kv_len], v[keys < kv_len], keys[keys < kv_len]
            z = torch.einsum("nhd,kd->hnk", q[q0:q0 + n, p * g:(p + 1) * g], k) / math.sqrt(d)
            hidden = keys[None] > pos0 + torch.arange(n, device=q.device)[:, None]
            z = z.masked_fill(hidden, -math.inf)
            norm = torch.logsumexp(z, -1)
            w = torch.exp(z - norm.masked_fill(norm == -math.inf, 0.0)[..., None])
            o[q0:q0 + n, p * g:(p + 1) * g] = torch.einsum("hnk,kd->nhd", w, v)
            lse[q0:q0 + n, p * g:(p + 1) * g] = norm.T
    return o, lse


def _turned(s, x, inverse=False):
    """x with its pairs taken as complex numbers and turned, in fp64."""
    case, x = s["case"], x.double().clone()
    r = case["rot"]
    turns, a = _freqs(r, case["scaling"], case["factor"])
    phase = torch.remainder(s["positions"].double()[:, None] * turns.to(x.device), 1.0) * (2 * math.pi)
    z = torch.polar(torch.full_like(phase, a), -phase if inverse else phase)[:, None]
    if case["layout"] == "half":
        y = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * z
        x[..., :r // 2], x[..., r // 2:r] = y.real, y.imag
    else:
        x[..., :r] = torch.view_as_real(torch.view_as_complex(x[..., :r].unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
    return x


def _to_e4m3(x):
    """The e4m3 value nearest to each x, ties to even, saturating at 448."""
    x = x.clamp(-448, 448)
    step = 2.0 ** (torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step
