"""How exact the 8-bit cache's attention is over fp32 rows.  The bound of the other tests counts every
rounding at its worst, which grows with head dim, scores and length until a kernel that lost half of a
query's bits would pass.  Here the error of a row (all elements of a head's output) is taken relative to
u = sqrt(sum_p |w_p v_p|^2), what independent errors of the weights w_p add up to.  (Not element by element: with scores far
apart one position has nearly all the weight, and where its code is 0 an element consists of weights as small as 2^-70, which
the fixed step of the weights rightly takes out.)

The limit for scores of size 1, 2^-19 in the mean square, lies between two counts.  What has to be there: queries to
2^-22 of their largest element (2 fp16 terms) or better, sums of a score in fp32 (eight or sixteen truncations of 2^-24 of its
size), the exponent's argument and the exponential (2^-22), weights to 2^-22 or a fixed step of 2^-28 of the
largest, sums of a tile's output in fp32 (sixteen truncations): each some 1e-7, under 1e-6 together.
What would be a loss: queries of 16 bits (2^-17 of the largest element, 2.7 times the mean one: 2^-17 x 2.7 / sqrt(3) = 1.2e-5 of a
score of size 1), one fp16 term of a query or weight (2^-12 / sqrt(3) = 1.4e-4), weights of 16 bits (a step of 2^-12).
With scores sixteen times as large their errors are too, but few positions have the weight, with errors much alike: four
times the limit, of which the models stay under a tenth.  Both counts are computed below in a model of the arithmetic, on the CPU."""
import math

import numpy as np
import pytest

from tests import branch_util as bu
from tests import kv8_util as ku

LIMIT = {1: 2.0 ** -19, 16: 2.0 ** -17}  # by the size of the scores


# ------------------------------------------------- a model of the arithmetic
def f32(x):
    return np.float32(x).astype(np.float64)


def f16(x):
    return np.float16(x).astype(np.float64)


def truncated(x):
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(m * 2.0 ** 24) / 2.0 ** 24, e)


def product(a, b, step, acc=0.0):
    """acc + a b^T, `step` inner elements at a time, truncated to fp32 after each."""
    for k in range(0, a.shape[1], step):
        acc = truncated(acc + a[:, k:k + step] @ b[:, k:k + step].T)
    return acc


def fixed(x, bits):
    """Whole numbers (32 bits) without their lowest 32 - bits."""
    return np.round(x * 2.0 ** (bits - 32)) * 2.0 ** (32 - bits)


def by_digits(a, b):
    """a b^T for whole numbers a of up to 32 bits, by their eight hexadecimal digits."""
    sign, left, out = np.sign(a), np.abs(a), 0.0
    for n in range(8):  # the lowest first
        digit = np.mod(left, 16.0)
        left = np.floor(left / 16.0)
        out = f32(out / 16.0 + product(sign * digit, b, 32))
    return out * 16.0 ** 7


def few(rng, q, k, kp, v, vp, q_bits=32, w_bits=32):
    """The kernel of few rows.  k, v: codes' values; kp, vp: their powers' exponents, one for each position."""
    c = f32(math.log2(math.e) / math.sqrt(q.shape[1]))
    top = np.exp2(np.frexp(np.abs(q).max(1, keepdims=True))[1])
    s = by_digits(fixed(np.minimum(np.round(np.abs(q) / top * 2.0 ** 32), 2.0 ** 32 - 1), q_bits) * np.sign(q), k) * top * 2.0 ** -32
    x = f32(s * f32(c * np.exp2(kp))[None])
    base, sums, out = np.full((len(q), 1), -1e30), np.zeros((len(q), 128)), np.zeros((len(q), v.shape[1]))
    for t in range(0, len(k), 128):
        xt, e = x[:, t:t + 128], vp[None, t:t + 128]
        w = np.exp2(np.minimum(f32(xt - base), 1000.0))
        if (w * np.exp2(e) > 8).any():
            new = np.maximum(base, f32(xt + e).max(1, keepdims=True))
            corr = f32(np.exp2(np.maximum(base - new, -2000.0)))
            base, sums, out = new, f32(sums * corr), f32(out * corr)
        w = f32(np.exp2(f32(xt - base)) * (1 + rng.uniform(-1, 1, xt.shape) * 2.0 ** -22))
        sums[:, :w.shape[1]] = f32(sums[:, :w.shape[1]] + w)
        out = f32(out + by_digits(fixed(np.round(w * np.exp2(e) * 2.0 ** 28), w_bits), v[t:t + 128].T) * 2.0 ** -28)
    return out / f32(sums.sum(1, keepdims=True))


def terms(x, n, cut):
    """x as n fp16 terms; cut: the first has its upper 11 bits."""
    hi = x
    if cut and n > 1:
        m, e = np.frexp(x)
        hi = np.ldexp(np.trunc(m * 2.0 ** 11) / 2.0 ** 11, e)
    return [f16(hi)] + ([f16(f32(x - (hi if cut else f16(hi))))] if n > 1 else [])


def wide(rng, q, k, kp, v, vp, q_terms=2, w_terms=2):
    """The kernel of many rows."""
    c = f32(math.log2(math.e) / math.sqrt(q.shape[1]))
    top = np.exp2(np.frexp(np.abs(q).max(1, keepdims=True))[1] - 15.0)
    s = 0.0
    for term in reversed(terms(q / top, q_terms, False)):
        s = product(term, k, 16, s)
    scale = f32(f32(c * top) * np.exp2(kp)[None])
    groups = [[np.full((len(q), 1), -1e30), np.zeros((len(q), 1))] for _ in range(2)]  # of even and odd tiles: base, sum
    base, out = np.full((len(q), 1), -1e30), np.zeros((len(q), v.shape[1]))
    for t in range(0, len(k), 128):
        g = groups[t // 128 % 2]
        e = vp[None, t:t + 128]
        best = f32(s[:, t:t + 128] * scale[:, t:t + 128] + e).max(1, keepdims=True)
        new = np.where(best - g[0] > 15, np.ceil(best) - 8, g[0])
        g[1] = f32(g[1] * np.exp2(np.maximum(g[0] - new, -2000.0)))
        g[0] = new
        w = f32(np.exp2(f32(s[:, t:t + 128] * scale[:, t:t + 128] + f32(e - new))) * (1 + rng.uniform(-1, 1, (len(q), e.shape[1])) * 2.0 ** -22))
        g[1] = f32(g[1] + f32((w * np.exp2(-e)).sum(1, keepdims=True)))
        o = 0.0
        for term in reversed(terms(w, w_terms, True)):
            o = product(term, v[t:t + 128].T, 16, o)
        rise = new - base > 10
        out = np.where(rise, f32(out * np.exp2(np.clip(base - new, -2000.0, 0.0))), out)
        base = np.where(rise, new, base)
        out = f32(out + o * np.exp2(new - base))
    return out / sum(g[1] * np.exp2(np.maximum(g[0] - base, -2000.0)) for g in groups)


def case(rng, n, hd, scale):
    """16 queries; keys and values as E4M3 values and exponents of blocks of 16, with blocks of other sizes."""
    def rows():
        x = rng.standard_normal((-(-n // 16), 16, hd)) * np.exp(rng.standard_normal((-(-n // 16), 1, 1)) * 0.5)
        e = np.array([ku.power(float(np.abs(b).max())) - 127.0 for b in x])
        return ku.e4m3(x / np.exp2(e)[:, None, None]).reshape(-1, hd)[:n], np.repeat(e, 16)[:n]
    return (f32(rng.standard_normal((16, hd)) * scale), *rows(), *rows())


def rms(out, q, k, kp, v, vp):
    keys, vals = k * np.exp2(kp)[:, None], v * np.exp2(vp)[:, None]
    s = q @ keys.T / math.sqrt(q.shape[1])
    w = np.exp(s - s.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    return float(np.sqrt((((out - w @ vals) ** 2).sum(1) / (w ** 2 @ vals ** 2).sum(1)).mean()))


@pytest.mark.parametrize("scale", [1, 16])
@pytest.mark.parametrize("n,hd", [(9, 128), (140, 64), (2000, 128), (9000, 64)])
def test_the_limit_tells_the_kernels_from_ones_that_lose_bits(n, hd, scale):
    rng = np.random.default_rng(n + hd)
    c = case(rng, n, hd, scale)
    limit = LIMIT[scale]
    for model, worse in ((few, (dict(q_bits=16), dict(w_bits=16))), (wide, (dict(q_terms=1), dict(w_terms=1)))):
        assert rms(model(rng, *c), *c) < limit / 1.5, model
        for loss in worse:
            assert rms(model(rng, *c, **loss), *c) > limit, loss


# ------------------------------------------------------------- the kernels
CASES = [
    # tree, lens, rows, heads, kv heads, head dim; a few rows to a kv head
    (True, [7, 1, 300], [2, 1, 5], 2, 1, 128), (True, [131] * 3, [8] * 3, 16, 8, 128), (True, [9000], [8], 16, 8, 128),
    (False, [30000], [1], 8, 8, 64), (False, [500, 2000, 9000] * 30, [1] * 90, 4, 2, 128), (True, [9000] * 20, [4] * 20, 8, 2, 64),
    # many: shared by clusters, and filling the GPU; prompts and chunks
    (True, [300], [64], 4, 2, 128), (True, [9000], [64], 4, 2, 64), (True, [30000], [64], 16, 8, 128), (True, [2000] * 80, [64] * 80, 4, 2, 128),
    (False, [0], [700], 8, 4, 128), (False, [5000, 0], [300, 900], 4, 4, 64), (False, [100] * 40, [130] * 40, 8, 4, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("block", [16, 4, 1])
@pytest.mark.parametrize("scale", [1, 16])
@pytest.mark.parametrize("which", range(len(CASES)))
def test_attention_of_fp32_rows_holds_its_bits(which, scale, block):
    import torch
    from autoregressive_tts_decode_gb300 import build, q3tts
    build.build()
    tree, lens, rows, heads, kvh, hd = CASES[which]
    rng, page = np.random.default_rng(which), 16
    total = [a + b for a, b in zip(lens, rows)]
    pages, table = bu.page_table(rng, total, page)
    gen = torch.Generator(device="cuda").manual_seed(which)
    pool = torch.zeros((1, pages, 2, kvh, page, hd), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros((1, pages, 2, kvh, page // block), dtype=torch.uint8, device="cuda")
    tab = torch.from_numpy(table).cuda()
    k, v = (torch.randn((sum(total), kvh, hd), generator=gen, device="cuda") *
            torch.exp(0.5 * torch.randn((sum(total) // 16 + 1, kvh, 1), generator=gen, device="cuda")).repeat_interleave(16, 0)[:sum(total)]
            for _ in range(2))
    q3tts.kv8_write(pool, scales, 0, tab, ku.ints([0] * len(lens)), ku.ints(ku.starts(total)), k, v, max_rows=max(total))
    q = torch.randn((sum(rows), heads, hd), generator=gen, device="cuda") * scale
    start = ku.starts(rows)
    mt = bu.masks_tensor(sum((bu.tree_masks(bu.tree_parents(rng, n)) for n in rows), [])) if tree else None
    out = q3tts.kv8_attention(pool, scales, 0, tab, ku.ints(lens), ku.ints(start), q, masks=mt, max_rows=max(rows))
    two = torch.exp2(scales.double() - 127)
    sq = 0.0
    for s, (length, n) in enumerate(zip(lens, rows)):
        pos = torch.arange(length + n, device="cuda")
        at = tab[s].long()[pos // page], pos % page
        kv = pool[0, at[0], :, :, at[1]].double() * two[0, at[0], :, :, at[1] // block][..., None]  # [positions, 2, kv heads, hd]
        mine = slice(int(start[s]), int(start[s]) + n)
        if tree:
            sees = (pos < length) | (((mt[mine, None] >> (pos - length).clamp(0, 63)) & 1) != 0)
        else:
            sees = pos[None] - length <= torch.arange(n, device="cuda")[:, None]
        for h in range(heads):
            keys, vals = kv[:, 0, h // (heads // kvh)], kv[:, 1, h // (heads // kvh)]
            w = torch.softmax((q[mine, h].double() @ keys.T / math.sqrt(hd)).masked_fill(~sees, -math.inf), -1)
            sq += float((((out[mine, h].double() - w @ vals) ** 2).sum(-1) / (w ** 2 @ vals ** 2).sum(-1)).sum())
    off = math.sqrt(sq / (sum(rows) * heads))
    assert off < LIMIT[scale], off / LIMIT[scale]
