"""Shared helpers of the branching-decode tests: paged caches with NaN in every
unwritten word, random trees, and the operators' definitions in 64 bits."""
from __future__ import annotations

import math

import numpy as np


def page_table(rng, lens, page, spare=2):
    """(pages of the pool, int32 table): distinct pages in random order; entries
    past a sequence's last page point outside the pool."""
    need = [-(-n // page) for n in lens]
    pages = max(1, sum(need)) + spare
    perm = rng.permutation(pages)
    table = np.full((len(lens), max(need + [1])), 1 << 29, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    return pages, table


def paged_cache(rng, lens, page, layers, kv_heads, hd, dtype):
    """(pool, table) on the GPU: random keys and values in the sequences'
    positions, NaN everywhere else."""
    import torch
    pages, table = page_table(rng, lens, page)
    pool = torch.full((layers, pages, 2, kv_heads, page, hd), math.nan, dtype=dtype, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 31)))
    for s, n in enumerate(lens):
        for j in range(-(-n // page)):
            rows = min(page, n - j * page)
            pool[:, table[s, j], :, :, :rows] = torch.randn((layers, 2, kv_heads, rows, hd), generator=gen,
                                                            device="cuda").to(dtype)
    return pool, torch.from_numpy(table).cuda()


def tree_parents(rng, n):
    return [-1 if i == 0 else int(rng.integers(-1, i)) for i in range(n)]


def tree_masks(parents):
    out = []
    for i, p in enumerate(parents):
        out.append((1 << i) | (out[p] if p >= 0 else 0))
    return out


def masks_tensor(masks):
    import torch
    return torch.from_numpy(np.array(masks, np.uint64).view(np.int64)).cuda()


def tree_reference(pool, layer, table, lens, nodes, masks, q):
    """(output, bound) in 64 bits.  The bound counts roundings: probabilities
    carried as three bf16 terms (24 bits: 2^-24 of each), the exponential's own
    error (2^-21), the score's (products and sums in fp32, 2^-24 each), and fp32
    sums over the positions."""
    import torch
    rows, heads, hd = q.shape
    kvh, page = pool.shape[3], pool.shape[4]
    rep = heads // kvh
    out = torch.zeros((rows, heads, hd), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    r0 = 0
    for s, (length, n) in enumerate(zip(lens, nodes)):
        if n == 0:
            continue
        total = length + n
        pos = torch.arange(total, device="cuda")
        pg, slot = table[s].long()[pos // page], pos % page
        k, v = (pool[layer, pg, j, :, slot].double() for j in (0, 1))
        ok = torch.ones((n, total), dtype=torch.bool, device="cuda")
        for i in range(n):
            for j in range(n):
                ok[i, length + j] = bool((masks[r0 + i] >> j) & 1)
        for h in range(heads):
            qs, kh, vh = q[r0:r0 + n, h].double(), k[:, h // rep], v[:, h // rep]
            sc = (qs @ kh.T / math.sqrt(hd)).masked_fill(~ok, -math.inf)
            p = torch.softmax(sc, -1)
            p = torch.where(ok.any(-1, keepdim=True), p, torch.zeros_like(p))
            size = (qs.abs() @ kh.abs().T / math.sqrt(hd)).masked_fill(~ok, 0.0).amax(-1, keepdim=True)
            err = 2.0 ** -24 + 2.0 ** -21 + 2 * (hd + 8) * 2.0 ** -24 * size + total * 2.0 ** -24
            out[r0:r0 + n, h] = p @ vh
            tol[r0:r0 + n, h] = (p @ vh.abs()) * err
        r0 += n
    return out, tol + 1e-30


def beam_scores(logits, scores, history=None, finished=None, eos=-1, special=0, penalty=1.0):
    """Candidate scores [groups, beams, vocab] in 64 bits (numpy; the logits'
    penalty in fp32, as the sampler's)."""
    x = np.asarray(logits, np.float32).copy()
    if history is not None and penalty != 1.0:
        pen = np.float32(penalty)
        x = np.where(np.asarray(history) != 0, np.where(x > 0, x / pen, x * pen), x)
    v = np.arange(x.shape[-1])
    if special > 0:
        x[..., (v >= special) & (v != eos)] = -np.inf
    x[np.isnan(x)] = -np.inf
    y = x.astype(np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        top = y.max(-1, keepdims=True)
        d = np.where(y == top, 0.0, y - top)
        d[np.isneginf(y)] = -np.inf
        z = np.log(np.exp(d).sum(-1, keepdims=True))
        sc = np.asarray(scores, np.float64)[..., None] + (d - z)
    sc[np.isnan(sc)] = -np.inf
    if finished is not None:
        for g, b in zip(*np.nonzero(np.asarray(finished))):
            sc[g, b] = -np.inf
            sc[g, b, eos] = np.float64(np.asarray(scores)[g, b])
    return sc, x


def beam_reference(logits, scores, k, **kw):
    """tokens, parents, scores by the documented order."""
    sc, x = beam_scores(logits, scores, **kw)
    g, b, v = sc.shape
    tok, par, best = np.full((g, k), -1, np.int32), np.zeros((g, k), np.int32), np.full((g, k), -np.inf)
    for i in range(g):
        beam, code = np.meshgrid(np.arange(b), np.arange(v), indexing="ij")
        order = np.lexsort((code.ravel(), -x[i].ravel(), beam.ravel(), -sc[i].ravel()))[:k]
        for j, at in enumerate(order):
            if sc[i].ravel()[at] > -np.inf:
                tok[i, j], par[i, j], best[i, j] = code.ravel()[at], beam.ravel()[at], sc[i].ravel()[at]
    return tok, par, best
