"""Shared helpers of the 8-bit cache's tests: caches whose unwritten codes and
powers are NaN, and the operators' definitions in 64 bits."""
from __future__ import annotations

import math

import numpy as np

from tests import branch_util as bu

NAN = 0x7F  # an E4M3 code
VALUES = np.array([(-1.0 if c & 128 else 1.0) * ((8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10) if c & 120 else (c & 7) * 2.0 ** -9)
                   if c & 127 != NAN else math.nan for c in range(256)])  # of the 256 codes


def e4m3(x):
    """x (numpy, 64 bits, at most 448 in size) rounded to E4M3, ties to even."""
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(x)
        step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
        return np.round(x / step) * step


def power(top):
    """The byte of a block whose largest finite magnitude is top (a Python float)."""
    b = 0
    while top > 448.0 * 2.0 ** (b - 127):
        b += 1
    return b


def cache(rng, lens, page, block, layers, kv_heads, hd, lo=121, hi=130):
    """(codes uint8, powers uint8, int32 table), numpy: random codes in the sequences'
    positions, powers lo .. hi in their blocks, NaN everywhere else, page ids outside the
    pool past a sequence's last one."""
    pages, table = bu.page_table(rng, lens, page)
    codes = np.full((layers, pages, 2, kv_heads, page, hd), NAN, np.uint8)
    powers = np.full((layers, pages, 2, kv_heads, page // block), 255, np.uint8)
    for s, n in enumerate(lens):
        for j in range(-(-n // page)):
            rows = min(page, n - j * page)
            c = rng.integers(0, 256, (layers, 2, kv_heads, rows, hd), np.uint8)
            codes[:, table[s, j], :, :, :rows] = np.where(c & 127 == NAN, 0, c)
            used = -(-rows // block)
            powers[:, table[s, j], :, :, :used] = rng.integers(lo, hi + 1, (layers, 2, kv_heads, used))
    return codes, powers, table


def to_gpu(codes, powers, table):
    import torch
    return (torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(powers).cuda().view(torch.float8_e8m0fnu),
            torch.from_numpy(table).cuda())


def ints(v):
    import torch
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def starts(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


def write_reference(codes, powers, layer, table, lens, rows, k, v):
    """Values (float64) and powers after the write; k and v numpy float64 [rows, kv heads, hd]."""
    page, blocks = codes.shape[4], powers.shape[4]
    block = page // blocks
    val, pw = VALUES[codes], powers.copy()
    r0 = 0
    for s, (length, n) in enumerate(zip(lens, rows)):
        for first in range(length // block * block, length + n, block):
            a, b = max(first, length), min(first + block, length + n)
            if a >= b:
                continue
            pg, sub, base = table[s, first // page], first % page // block, first % page
            for j, x in enumerate((k, v)):
                for h in range(codes.shape[3]):
                    new = x[r0 + a - length:r0 + b - length, h]
                    fin = np.isfinite(new)
                    byte = power(float(np.abs(new[fin]).max()) if fin.any() else 0.0)
                    if a > first:
                        before = int(pw[layer, pg, j, h, sub])
                        byte = max(byte, before)
                        if byte > before:
                            at = (layer, pg, j, h, slice(base, base + a - first))
                            val[at] = e4m3(val[at] * 2.0 ** (before - byte))
                    pw[layer, pg, j, h, sub] = byte
                    val[layer, pg, j, h, base + a - first:base + b - first] = np.where(
                        fin, e4m3(np.where(fin, new, 0.0) * 2.0 ** (127 - byte)), math.nan)
        r0 += n
    return val, pw


def values(codes, powers, layer, table, s, pos):
    """Codes' values and powers (float64) of sequence s's positions: [2, positions, kv heads, hd], [2, positions, kv heads]."""
    page, block = codes.shape[4], codes.shape[4] // powers.shape[4]
    pos = np.asarray(pos, np.int64)
    pg, slot = table[s, pos // page], pos % page
    c = np.stack([VALUES[codes[layer, pg, j, :, slot]] for j in (0, 1)])
    p = np.stack([np.exp2(powers[layer, pg, j, :, slot // block].astype(np.float64) - 127) for j in (0, 1)])
    return c, p


def attention_reference(codes, powers, layer, table, lens, rows, masks, q):
    """(output, bound) in 64 bits on the GPU; q fp32 or bf16.

    The bound counts roundings.  Scores: the query in fixed point of at least 24 bits below
    its largest element, products and sums in fp32 (2^-24 each, 2 hd of them).  Weights: the exponential's error
    (2^-21), fp32 sums over the positions (2^-24 each), two fp16 terms (2^-22) or a fixed point whose step is at most 2^-27
    of the largest weight x value power; with bf16 rows one fp16 term (half a step: 2^-11).  The output: half a step of its
    type."""
    import torch
    n_rows, heads, hd = q.shape
    rep = heads // codes.shape[3]
    half = q.dtype == torch.bfloat16
    out = torch.zeros((n_rows, heads, hd), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    r0 = 0
    for s, (length, n) in enumerate(zip(lens, rows)):
        if n == 0:
            continue
        total = length + n
        c, p = values(codes, powers, layer, table, s, np.arange(total))
        c, p = torch.from_numpy(c).cuda(), torch.from_numpy(p).cuda()
        ok = torch.ones((n, total), dtype=torch.bool, device="cuda")
        if masks is None:
            ok[:, length:] = torch.ones((n, n), device="cuda").tril() > 0
        else:
            for i in range(n):
                for j in range(n):
                    ok[i, length + j] = bool((masks[r0 + i] >> j) & 1)
        any_seen = ok.any(-1, keepdim=True)
        # what no row sees may be NaN: taken out of the products
        seen = ok.any(0)
        c = torch.where(seen[None, :, None, None], c, 0.0)
        p = torch.where(seen[None, :, None], p, 0.0)
        for h in range(heads):
            g = h // rep
            qs, kh, vh = q[r0:r0 + n, h].double(), c[0, :, g] * p[0, :, g, None], c[1, :, g] * p[1, :, g, None]
            sc = (qs @ kh.T / math.sqrt(hd)).masked_fill(~ok, -math.inf)
            w = torch.where(any_seen, torch.softmax(sc, -1), 0.0)
            size = (qs.abs() @ kh.abs().T / math.sqrt(hd)).masked_fill(~ok, 0.0).amax(-1, keepdim=True)
            fixed = qs.abs().amax(-1, keepdim=True) * 2.0 ** -24 * (
                kh.abs().sum(-1)[None].masked_fill(~ok, 0.0).amax(-1, keepdim=True) / math.sqrt(hd))
            err = 2.0 ** -21 + 2.0 ** -22 + 2 * fixed + 2 * (2 * hd + 8) * 2.0 ** -24 * size + total * 2.0 ** -24
            if half:
                err = err + 2.0 ** -11
            step = 2.0 ** -27 * (w * p[1, :, g][None]).amax(-1, keepdim=True)
            o = w @ vh
            out[r0:r0 + n, h] = o
            t = (w @ vh.abs()) * err + step * (ok.double() @ c[1, :, g].abs())
            tol[r0:r0 + n, h] = t + (o.abs() + t) * (2.0 ** -8 if half else 2.0 ** -24)
        r0 += n
    return out, tol + 1e-30
