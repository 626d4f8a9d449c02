"""Trees of drafts and latent caches for the tests: inputs, and the attention by
its definition in 64 bits."""
import numpy as np
import torch

PAGE = 128


def tree_mask(qo, rng, empty=0.1):
    """int32 [rows, 4] and the same as booleans [rows, 128]: ancestors and itself;
    a share of the rows see no draft, and bits of drafts that are not there are
    set at random."""
    rows = []
    for q in qo:
        seen = np.zeros((q, 128), bool)
        for i in range(q):
            parent = rng.integers(-1, i)
            if parent >= 0:
                seen[i] = seen[parent]
            seen[i, i] = True
        seen[rng.random(q) < empty] = False
        rows.append(seen)
    seen = np.concatenate(rows)
    noise = rng.random(seen.shape) < 0.5
    there = np.concatenate([np.broadcast_to(np.arange(128) < q, (q, 128)) for q in qo])
    bits = np.where(there, seen, noise).reshape(-1, 4, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)
    return bits.sum(-1).astype(np.uint32).view(np.int32), seen


def chain_mask(qo):
    """The mask of causal rows."""
    seen = np.concatenate([np.tril(np.ones((q, 128), bool)) for q in qo])
    bits = seen.reshape(-1, 4, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)
    return bits.sum(-1).astype(np.uint32).view(np.int32)


def tiles(qo, kv):
    """(first row, rows, position of the first row, kv_len, first page-table entry, blocks) of each tile."""
    out, q0, base = [], 0, 0
    for q, k in zip(qo, kv):
        for r in range(0, q, PAGE):
            n = min(PAGE, q - r)
            out.append((q0 + r, n, k - q + r, k, base, (k - q + r + n - 1) // PAGE + 1))
        q0, base = q0 + q, base + (k + PAGE - 1) // PAGE
    return out


def selection(qo, kv, hp, topk, rng, irregular=True):
    """Distinct blocks in random order with -1 among them; some rows select nothing,
    some leave the diagonal block out."""
    tl = tiles(qo, kv)
    idx = np.full((len(tl), hp, topk), -1, np.int32)
    for t, tile in enumerate(tl):
        for h in range(hp):
            sel = rng.permutation(tile[5])[:topk]
            idx[t, h, :len(sel)] = sel
            if irregular:
                idx[t, h] = idx[t, h][rng.permutation(topk)]
                if (t * hp + h) % 7 == 5:
                    idx[t, h] = -1
    return idx


def attend(q, k_of, v_of, qo, kv, idx, scale, seen=None, groups=None):
    """out and lse in fp64, with what bounds their errors: A = sum w |v| / sum w by
    output, B = the largest scale * sum |q| |k| of a seen pair by (row, head).
    k_of, v_of(entry of the page table, proxy head): fp64 [128, width] blocks;
    seen: bool [rows, 128] over the drafts (None: causal)."""
    hp = idx.shape[1]
    g = q.shape[1] // hp
    wide = v_of(0, 0).shape[1]
    dev = q.device
    o = torch.zeros((q.shape[0], q.shape[1], wide), dtype=torch.float64, device=dev)
    a, b = torch.zeros_like(o), torch.zeros(q.shape[:2], dtype=torch.float64, device=dev)
    lse = torch.full(q.shape[:2], -np.inf, dtype=torch.float64, device=dev)
    for (q0, n, pos0, kv_len, base, _), sel in zip(tiles(qo, kv), idx):
        for h in range(hp):
            blocks = [int(j) for j in sel[h] if j >= 0]
            if not blocks:
                continue
            keys = np.concatenate([np.arange(j * PAGE, (j + 1) * PAGE) for j in blocks])
            e = keys[None] - pos0 - np.zeros((n, 1), np.int64)
            if seen is None:
                vis = e <= np.arange(n)[:, None]
            else:
                vis = (e < 0) | ((e < 128) & np.take_along_axis(seen[q0:q0 + n], np.clip(e, 0, 127), 1))
            vis &= keys < kv_len
            vis = torch.from_numpy(vis).to(dev)
            any_row = vis.any(0)
            k = torch.cat([k_of(base + j, h) for j in blocks])
            v = torch.cat([v_of(base + j, h) for j in blocks])
            k, v = (torch.where(any_row[:, None], x, 0.0) for x in (k, v))
            x = q[q0:q0 + n, h * g:(h + 1) * g].double()
            z = torch.einsum("nhd,kd->hnk", x, k) * scale
            z = z.masked_fill(~vis, -np.inf)
            norm = torch.logsumexp(z, -1)
            w = torch.exp(z - norm.masked_fill(norm == -np.inf, 0.0)[..., None])
            o[q0:q0 + n, h * g:(h + 1) * g] = torch.einsum("hnk,kd->nhd", w, v)
            a[q0:q0 + n, h * g:(h + 1) * g] = torch.einsum("hnk,kd->nhd", w, v.abs())
            lse[q0:q0 + n, h * g:(h + 1) * g] = norm.T
            mag = torch.einsum("nhd,kd->hnk", x.abs(), k.abs()) * scale
            b[q0:q0 + n, h * g:(h + 1) * g] = mag.masked_fill(~vis, 0.0).amax(-1).T
    return o, lse, a, b


def check(out, lse, ref, width, kind, n_keys, room=0.0):
    """out (bf16) and lse (fp32) against attend()'s, by the roundings:
      - a logit is a sum of width / 16 products of 16 in fp32, each addition off by
        2^-22 of the largest partial sum at most, which B bounds: E = width / 16 *
        2^-22 * B + 2^-22 * B (the multiply-add that scales it), so a weight is off by 2 E
        relative, and the exponentials by 2^-22 each;
      - weights are rounded to bf16 (half a step 2^-8 relative) or, for e4m3 caches,
        to f16 (2^-11; below f16's normal range 2^-25 of the largest at most, which
        `room` takes: 2^-25 * keys * the largest |value|);
      - the result is rounded to bf16: 2^-8 of itself."""
    o, norm, a, b = ref
    assert out.dtype == torch.bfloat16 and not torch.isnan(out).any() and not torch.isnan(lse).any()
    e = (width / 16 + 1) * 2.0 ** -22 * b
    step = 2.0 ** -8 if kind in ("bf16", "latent") else 2.0 ** -11
    tol = ((step + 2.0 ** -20 + 2 * e)[..., None] * a + room) * (1 + 2.0 ** -8) + 2.0 ** -8 * o.abs() + 1e-30
    err = (out.double() - o).abs()
    assert (err <= tol).all(), "out off by %g of its bound" % (err / tol).max().item()
    empty = norm == -np.inf
    assert torch.equal(lse == -np.inf, empty) and (out[empty] == 0).all()
    # the sum of up to n weights in fp32: 2^-24 each addition, and the logarithm's own rounding
    # of m + log2 l, which is at most |m| + log2 n + 8
    lim = e + n_keys * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -22 * (norm.masked_fill(empty, 0.0).abs() + np.log(n_keys) + 8)
    assert ((lse.double() - norm).abs()[~empty] <= lim[~empty]).all()
