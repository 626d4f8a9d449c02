"""More operators of libmsa as cases to measure: attention for trees of drafted
tokens over the paged K/V cache, and a cache that holds one shared latent
vector a token: its append, attention over it in the absorbed form, and its
expansion into K and V pages.

Each operator has a plain form in elementary torch operations (fp32, angles
in fp64) and the library's call; `own` says which of the two run() takes.
"""
import math
import random

import torch

own = False

PAGE = 128


# ------------------------------------------------------------------- cases --

def listed():
    def batch(name, op, **kw):
        return dict(name=name, op=op, batch=1, rows=1, ctx=0, even=True, lens=0, topk=16) | kw

    def tree(name, **kw):
        return batch(name, "tree", hq=64, hkv=8, hp=8, d=128, kv="bf16") | kw

    def latent(name, op="latent", **kw):
        return batch(name, op, hq=64, hp=1, latent=512, rot=64, tree=False) | kw

    return [
        # a single user's 16 drafts checked in one step, at 131072 keys (latency)
        tree("verify 1 x 16 drafts", rows=16, ctx=131000, kv="e4m3_block"),
        # a serving batch with short trees
        tree("verify 32 x 8 drafts", batch=32, rows=8, ctx=32700),
        # trees of different sizes, three query heads a KV head, over a cache with one scale a head
        tree("verify ragged", batch=7, rows=61, ctx=9000, even=False, lens=3, hq=12, hkv=4, hp=4, d=64, kv="e4m3", topk=9),
        # a serving batch with wide trees
        tree("verify 32 x 64 drafts", batch=32, rows=64, ctx=32700, kv="e4m3_block"),
        # a single user's decode step at 131072 tokens (latency)
        latent("latent decode 1", ctx=131071),
        # a serving batch's decode step
        latent("latent decode 32", batch=32, ctx=32767),
        # draft trees of a ragged batch, a smaller latent and two selections a token
        latent("latent verify ragged", batch=6, rows=13, ctx=7000, even=False, lens=5, hq=20, hp=2, latent=256, rot=32,
               topk=11, tree=True),
        # a chunk of a prompt on top of a long context
        latent("latent chunk 512", rows=512, ctx=20000, hq=32),
        # one decode step of 32 sequences: a token's latent into pages that are partly filled (latency)
        latent("latent append decode", "append", batch=32, ctx=2000, even=False, lens=3),
        # the latents of a 32K prefill into an empty cache
        latent("latent append prefill 32K", "append", rows=32768),
        # the K and V of ragged prompts out of their latents, for the prefill attention
        latent("expand ragged", "expand", batch=5, rows=900, ctx=700, even=False, lens=7, hq=12, latent=256, rot=32) | dict(d=64),
        # the K and V of a 32K prompt out of its latents
        latent("expand 32K", "expand", rows=32768, hq=32) | dict(d=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "latent", "latent", "append", "expand"])
    case = dict(op=op, batch=_log_int(rng, 1, 32), even=False, lens=rng.randint(0, 10**6), topk=_log_int(rng, 1, 16))
    if op == "tree":
        hkv, m = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2])
        hq = hkv * m * rng.choice([1, 3, 4, 8 // m])
        return case | dict(rows=_log_int(rng, 1, 64), ctx=_log_int(rng, 1, 200000 // case["batch"]), hq=hq, hkv=hkv,
                           hp=hkv * m, d=rng.choice([64, 128]), kv=rng.choice(["bf16", "e4m3", "e4m3_block"]))
    case |= dict(latent=rng.choice([128, 256, 384, 512]), tree=False)
    if op == "latent":
        hp, tree = rng.choice([1, 1, 2, 4]), rng.random() < 0.4
        hq = hp * rng.choice([1, 5, 8, 16])
        rows = 1 if rng.random() < 0.4 else _log_int(rng, 2, min(64 if tree else 512, 8192 // (hq * case["batch"]) + 2))
        return case | dict(rows=rows, ctx=_log_int(rng, 1, 200000 // case["batch"]), hq=hq, hp=hp, tree=tree,
                           rot=rng.choice([16, 32, 48, 64]))
    case |= dict(rows=_log_int(rng, 1, 32768 // case["batch"]), hq=rng.randint(1, 32), hp=1, rot=rng.choice([16, 32, 64]))
    if op == "append":
        return case | dict(ctx=_log_int(rng, 1, 32768 // case["batch"]))
    half = max(1, case["rows"] // 2)                     # rows and context together cost no more than the largest case
    return case | dict(rows=half, ctx=_log_int(rng, 1, half), d=128 if case["rot"] == 64 else rng.choice([64, 128]))


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
    qo, kv = _lens(case)
    rows, op = sum(qo), case["op"]
    if op == "append":
        width = case["latent"] + case["rot"]
        return {"bytes": rows * (4 * width + 4), "flops": 3 * rows * case["rot"]}
    if op == "expand":
        keys, wide = sum(kv), case["latent"] + case["rot"]
        n = case["hq"] * (2 * case["d"] - case["rot"])
        return {"bytes": 2 * (keys * (wide + 2 * case["hq"] * case["d"]) + n * case["latent"]),
                "flops": 2 * keys * n * case["latent"]}
    pairs = sel = 0
    for q, k in zip(qo, kv):
        for r0 in range(0, q, PAGE):
            n = min(PAGE, q - r0)
            nb = min(case["topk"], (k - q + r0 + n - 1) // PAGE + 1)
            pairs += n * case["hq"] * nb * PAGE
            sel += nb * case["hp"]
    table = sum(_blocks(k) for k in kv)
    if op == "tree":
        per_page = 2 * PAGE * case["d"] * (2 if case["kv"] == "bf16" else 1)
        pages = min(sel, table * case["hkv"]) * per_page
        return {"bytes": rows * case["hq"] * (4 * case["d"] + 4) + pages + 4 * sel + 16 * rows,
                "flops": 4 * case["d"] * pairs}
    wide = case["latent"] + case["rot"]
    return {"bytes": rows * case["hq"] * (2 * wide + 2 * case["latent"] + 4) + min(sel, table) * PAGE * 2 * wide + 4 * sel,
            "flops": 2 * (wide + case["latent"]) * pairs}


# ------------------------------------------------------------------ inputs --

def _tables(qo, kv, gen):
    """What a serving program holds on the device beside the cache: the page
    table, each row's key position and place."""
    nb = [_blocks(k) for k in kv]
    num_pages = sum(nb) + 3
    table = torch.randperm(num_pages, generator=gen, device="cuda")[:sum(nb)].to(torch.int32)
    pos = torch.cat([torch.arange(k - q, k, device="cuda") for q, k in zip(qo, kv)])
    base, entry = 0, []
    for q, k, n in zip(qo, kv, nb):
        entry.append(base + torch.arange(k - q, k, device="cuda") // PAGE)
        base += n
    return dict(num_pages=num_pages, kv_indices=table, positions=pos.to(torch.int32),
                page=table.long()[torch.cat(entry)], slot=pos % PAGE)


def _trees(qo, gen):
    """Draft trees: bit b of word w of a row says that the row sees draft
    32 w + b of its sequence, an ancestor or itself.  About one row in nine is
    padding, which sees no draft."""
    cpu = torch.Generator().manual_seed(int(torch.randint(1 << 30, (1,), generator=gen, device="cuda")))
    seen = torch.zeros((sum(qo), PAGE), dtype=torch.bool)
    r0 = 0
    for q in qo:
        parent = (torch.rand(q, generator=cpu) * (torch.arange(q) + 1)).long() - 1
        for i in range(q):
            if parent[i] >= 0:
                seen[r0 + i] = seen[r0 + parent[i]]
            seen[r0 + i, i] = True
        seen[r0:r0 + q][torch.rand(q, generator=cpu) < 0.11] = False
        r0 += q
    bits = seen.view(-1, 4, 32).long() << torch.arange(32)
    words = bits.sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).cuda()


def _select(case, s, qo, kv, gen):
    """Tiles of 128 query rows, and a selection for each (tile, proxy head): the
    diagonal block and other blocks up to it, ascending, padded with -1."""
    tiles, q0, base = [], 0, 0
    for q, k in zip(qo, kv):
        for r in range(0, q, PAGE):
            n = min(PAGE, q - r)
            tiles.append((q0 + r, n, k - q + r, k, base, (k - q + r + n - 1) // PAGE + 1))
        q0, base = q0 + q, base + _blocks(k)
    s["tiles"] = torch.tensor(tiles, device="cuda")
    s["widest"] = max(t[1] for t in tiles)
    nvp, topk = s["tiles"][:, 5], case["topk"]
    wide = max(topk, max(t[5] for t in tiles))
    j = torch.arange(wide, device="cuda")
    score = torch.rand((len(tiles), case["hp"], wide), generator=gen, device="cuda")
    score = torch.where(j == nvp[:, None, None] - 1, 2.0, torch.where(j < nvp[:, None, None], score, -1.0))
    top, at = score.topk(topk, dim=-1)
    at = torch.where(top < 0, wide, at).sort(-1).values
    s["idx"] = torch.where(at == wide, -1, at).to(torch.int32).contiguous()


def _after_last(s, kv, pages, value):
    """What was never written behind a sequence's last key holds any bytes, NaN among them."""
    base = 0
    for i, k in enumerate(kv):
        base += _blocks(k)
        if i < 64:
            pages[s["kv_indices"][base - 1].long(), :, (k - 1) % PAGE + 1:] = value


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 2 + 1)
    qo, kv = _lens(case)
    op, rows = case["op"], sum(qo)
    s = dict(case=case) | _tables(qo, kv, gen)
    p = s["num_pages"]
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    if own:
        from block_sparse_long_proxy_gb300 import msa
    if op == "tree":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        _select(case, s, qo, kv, gen)
        s["mask"] = _trees(qo, gen)
        s["q"] = rand(rows, hq, d).to(torch.bfloat16)
        shape = (p, hkv, PAGE, d)
        for n, mean in (("k", -8), ("v", -7)):
            if case["kv"] == "bf16":
                s[n + "_pages"], s[n + "_scale"] = rand(*shape).to(torch.bfloat16), None
                _after_last(s, kv, s[n + "_pages"], math.nan)
                continue
            codes = rand(*shape).mul_(110.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
            _after_last(s, kv, codes.view(torch.uint8), 0x7F)
            one = 0.01 * (1 + torch.rand(hkv, generator=gen, device="cuda"))   # measured by calibration
            two = torch.exp2(torch.randint(mean - 1, mean + 2, (p, hkv), generator=gen, device="cuda").float())
            s[n + "_pages"], s[n + "_scale"] = codes, one if case["kv"] == "e4m3" else two
        if own:
            s["plan"] = msa.Plan(qo, kv, hq, hkv, case["hp"], d, 64, case["topk"], p, kv_dtype=case["kv"])
        return s
    latent, rot = case["latent"], case["rot"]
    if op == "append":
        # the latent and the key part that turns, as one projection's rows
        wide = rand(rows, latent + rot).to(torch.bfloat16)
        s["c"], s["kr"] = wide[:, None, :latent], wide[:, None, latent:]
        s["latent_pages"] = rand(p, 1, PAGE, latent + rot).to(torch.bfloat16)
        s["turns"] = (10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot) / (2 * math.pi)).cuda()
        if own:
            s["plan"], s["rope"] = msa.Plan(qo, kv, case["hq"], 1, 1, 128, 64, 1, p), msa.Rope(rot)
        return s
    s["latent_pages"] = rand(p, 1, PAGE, latent + rot).to(torch.bfloat16)
    _after_last(s, kv, s["latent_pages"], math.nan)
    if op == "expand":
        h, d = case["hq"], case["d"]
        s["w_k"], s["w_v"] = ((rand(h, n, latent) / math.sqrt(latent)).to(torch.bfloat16) for n in (d - rot, d))
        s["k_pages"], s["v_pages"] = (rand(p, h, PAGE, d).to(torch.bfloat16) for _ in range(2))
        nb = [_blocks(k) for k in kv]
        s["valid"] = torch.cat([(k - PAGE * torch.arange(n, device="cuda")).clamp(max=PAGE) for k, n in zip(kv, nb)])
        if own:
            s["plan"] = msa.Plan(qo, kv, h, h, h, d, 64, 1, p)
        return s
    _select(case, s, qo, kv, gen)
    s["mask"] = _trees(qo, gen) if case["tree"] else None
    s["q"] = (rand(rows, case["hq"], latent + rot) * 1.5).to(torch.bfloat16)
    s["scale"] = (latent + rot) ** -0.5
    if own:
        s["plan"] = msa.Plan(qo, kv, case["hq"], 1, case["hp"], 128, 64, case["topk"], p)
    return s


# --------------------------------------------------------------------- run --

def run(s):
    op, case = s["case"]["op"], s["case"]
    if op == "tree":
        if own:
            return s["plan"].tree_attn(s["q"], s["k_pages"], s["v_pages"], s["kv_indices"], s["idx"], s["mask"],
                                       k_scale=s["k_scale"], v_scale=s["v_scale"])
        at, there = _picked(s, case["hp"] // case["hkv"])
        k, v = _values(s, "k", at), _values(s, "v", at)
        return _attend(s, k, torch.where(there, v, 0.0), 1 / math.sqrt(case["d"]))
    if op == "latent":
        if own:
            return s["plan"].latent_attn(s["q"], s["latent_pages"], s["kv_indices"], s["idx"], case["rot"], s["scale"],
                                         tree_mask=s["mask"])
        (page, _), there = _picked(s, case["hp"])
        c = s["latent_pages"][page, 0].float()
        return _attend(s, c, torch.where(there, c[..., :case["latent"]], 0.0), s["scale"])
    if op == "append":
        if own:
            s["plan"].latent_append(s["c"], s["kr"], s["latent_pages"], s["kv_indices"], rope=s["rope"],
                                    positions=s["positions"])
        else:
            row = torch.cat((s["c"], _rotate(s, s["kr"]).to(torch.bfloat16)), -1)
            s["latent_pages"][s["page"], 0, s["slot"]] = row[:, 0]
        return s["latent_pages"]
    if own:
        s["plan"].latent_expand(s["latent_pages"], s["w_k"], s["w_v"], s["kv_indices"], s["k_pages"], s["v_pages"])
    else:
        page = s["kv_indices"].long()
        c = s["latent_pages"][page, 0].float()
        latent, h = case["latent"], case["hq"]
        c = torch.where(torch.arange(PAGE, device=c.device)[:, None] < s["valid"][:, None, None], c, 0.0)
        parts = [torch.matmul(c[:, None, :, :latent], s[w].float().transpose(1, 2)) for w in ("w_k", "w_v")]
        k = torch.cat((parts[0], c[:, None, :, latent:].expand(-1, h, -1, -1)), -1)
        good = (torch.arange(PAGE, device=c.device) < s["valid"][:, None])[:, None, :, None]
        for pages, x in ((s["k_pages"], k), (s["v_pages"], parts[1])):
            pages[page] = torch.where(good, x.to(torch.bfloat16), pages[page])
    return s["k_pages"], s["v_pages"]


def _rotate(s, x):
    """x [rows, 1, rot] with its pairs (i, i + rot / 2) turned, by angles taken in fp64."""
    turns = s["positions"].double()[:, None] * s["turns"]
    angle = (turns - torch.floor(turns)) * (2 * math.pi)
    c, sn = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = x.float().chunk(2, -1)
    return torch.cat((a * c - b * sn, b * c + a * sn), -1)


def _picked(s, per_head):
    """Where the selected blocks lie, (page, KV head) for [tiles, proxy heads,
    topk], and which of their keys are the sequence's."""
    idx, tiles = s["idx"].long(), s["tiles"]
    page = s["kv_indices"].long()[tiles[:, 4, None, None] + idx.clamp(min=0)]
    head = torch.arange(idx.shape[1], device=idx.device) // per_head
    key = idx[..., None] * PAGE + torch.arange(PAGE, device=idx.device)
    there = (idx[..., None] >= 0) & (key < tiles[:, 3, None, None, None])
    return (page, head[None, :, None]), there[..., None]


def _values(s, n, at):
    """K or V blocks in fp32, by their scales."""
    pages, scale = s[n + "_pages"], s[n + "_scale"]
    if scale is None:
        return pages[at].float()
    x = pages.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    by = scale[at[1]] if scale.dim() == 1 else scale[at]
    return x * by[..., None, None]


def _attend(s, k, v, scale):
    """Every (tile, proxy head) at once: its rows against its blocks k and v
    [tiles, proxy heads, topk, 128, width]."""
    q, idx, tiles, mask = s["q"], s["idx"].long(), s["tiles"], s["mask"]
    nt, hp, topk = idx.shape
    g = q.shape[1] // hp
    r = torch.arange(s["widest"], device=q.device)
    row = (tiles[:, 0, None] + r).clamp(max=q.shape[0] - 1)
    x = q.float()[row].unflatten(2, (hp, g)).permute(0, 2, 3, 1, 4).reshape(nt * hp, g * len(r), -1)
    sc = torch.bmm(x, k.reshape(nt * hp, topk * PAGE, -1).transpose(1, 2)).reshape(nt, hp, g, len(r), -1) * scale
    key = (idx[..., None] * PAGE + torch.arange(PAGE, device=q.device)).reshape(nt, hp, 1, -1)
    valid = (key >= 0) & (key < tiles[:, 3, None, None, None])
    if mask is None:
        seen = key <= (tiles[:, 2, None] + r)[:, None, :, None]
    else:
        draft = key - tiles[:, 2, None, None, None]
        word, bit = draft.clamp(0, PAGE - 1) // 32, draft.clamp(0, PAGE - 1) % 32
        words = mask[row][:, None].expand(-1, hp, -1, -1)
        seen = (draft < 0) | ((words.gather(3, word.expand(-1, -1, len(r), -1)) >> bit) & 1).bool()
    sc = torch.where((valid & seen)[:, :, None], sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    o = torch.bmm(e.reshape(nt * hp, -1, topk * PAGE), v.reshape(nt * hp, topk * PAGE, -1)).reshape(nt, hp, g, len(r), -1)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + torch.log(total))[..., 0]
    good = r < tiles[:, 1, None]
    rows = row[good]
    out = torch.empty((*q.shape[:2], o.shape[-1]), dtype=torch.bfloat16, device=q.device)
    out_lse = torch.empty(q.shape[:2], device=q.device)
    out[rows] = o.permute(0, 3, 1, 2, 4).reshape(nt, len(r), hp * g, -1)[good].to(torch.bfloat16)
    out_lse[rows] = lse.permute(0, 3, 1, 2).reshape(nt, len(r), hp * g)[good]
    return out, out_lse


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    """run()'s outputs from the definitions, in fp64."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "append":
        pages = s["latent_pages"].double()
        phase = torch.remainder(s["positions"].double()[:, None] * s["turns"], 1.0) * (2 * math.pi)
        half = case["rot"] // 2
        z = torch.complex(s["kr"][:, 0, :half].double(), s["kr"][:, 0, half:].double()) * torch.polar(torch.ones_like(phase), phase)
        pages[s["page"], 0, s["slot"]] = torch.cat((s["c"][:, 0].double(), z.real, z.imag), -1)
        return pages
    if op == "expand":
        out = [s["k_pages"].double(), s["v_pages"].double()]
        latent, nope = case["latent"], case["d"] - case["rot"]
        for i in range(len(s["kv_indices"])):
            page, n = int(s["kv_indices"][i]), int(s["valid"][i])
            c = s["latent_pages"][page, 0, :n].double()
            out[0][page, :, :n, :nope] = torch.einsum("tc,hnc->htn", c[:, :latent], s["w_k"].double())
            out[0][page, :, :n, nope:] = c[:, latent:]
            out[1][page, :, :n] = torch.einsum("tc,hnc->htn", c[:, :latent], s["w_v"].double())
        return tuple(out)
    # attention: one tile and proxy head after the other
    q, dev, wide = s["q"].double(), s["q"].device, case["latent"] if op == "latent" else case["d"]
    o = torch.zeros((*q.shape[:2], wide), dtype=torch.float64, device=dev)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=dev)
    hp = case["hp"]
    g = case["hq"] // hp
    scale = s["scale"] if op == "latent" else 1 / math.sqrt(case["d"])
    for (q0, n, pos0, kv_len, base, _), sel in zip(s["tiles"].tolist(), s["idx"].tolist()):
        words = s["mask"][q0:q0 + n].tolist() if s["mask"] is not None else None
        for h in range(hp):
            blocks = [j for j in sel[h] if j >= 0]
            if not blocks:
                continue
            at = s["kv_indices"].long()[torch.tensor(blocks, device=dev) + base]
            keys = torch.cat([torch.arange(j * PAGE, (j + 1) * PAGE) for j in blocks])
            keep = keys < kv_len
            keys = keys[keep]
            if op == "latent":
                k = s["latent_pages"][at, 0].double().flatten(0, 1)[keep.to(dev)]
                v = k[:, :wide]
            else:
                kv_head, k, v = h // (hp // case["hkv"]), None, None
                for name in ("k", "v"):
                    x, sc = s[name + "_pages"], s[name + "_scale"]
                    x = x[at, kv_head].double() if sc is None else x.view(torch.uint8)[at, kv_head].view(torch.float8_e4m3fn).double()
                    if sc is not None:
                        x = x * (sc[kv_head].double() if sc.dim() == 1 else sc[at, kv_head].double()[:, None, None])
                    k, v = (x.flatten(0, 1)[keep.to(dev)], v) if name == "k" else (k, x.flatten(0, 1)[keep.to(dev)])
            draft = (keys - pos0).tolist()
            if words is None:
                hidden = keys[None] > pos0 + torch.arange(n)[:, None]
            else:
                old, table = (keys < pos0)[None].repeat(n, 1), torch.zeros((n, PAGE), dtype=torch.bool)
                for i in range(n):
                    table[i] = torch.tensor([words[i][b // 32] >> (b % 32) & 1 for b in range(PAGE)], dtype=torch.bool)
                hidden = ~(old | (table[:, torch.tensor(draft).clamp(0, PAGE - 1)] & ~old))
            z = torch.einsum("nhd,kd->hnk", q[q0:q0 + n, h * g:(h + 1) * g], k) * scale
            z = z.masked_fill(hidden.to(dev), -math.inf)
            norm = torch.logsumexp(z, -1)
            w = torch.exp(z - norm.masked_fill(norm == -math.inf, 0.0)[..., None])
            o[q0:q0 + n, h * g:(h + 1) * g] = torch.einsum("hnk,kd->nhd", w, v)
            lse[q0:q0 + n, h * g:(h + 1) * g] = norm.T
    return o, lse
