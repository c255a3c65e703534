"""How exact the tree attention is.  The bound of the other tests counts every
rounding at its worst, which grows with the length until a kernel that lost half of
its bits would pass.  Here the error of an output element is taken relative to
u = sqrt(sum_p (w_p v_p)^2), what independent errors of the weights w_p add up to:
its root mean square does not depend on how many positions share the weight.

The limit, 2^-20, lies between two counts.  Weights held as two bf16 terms are off by
up to 2^-18 of their binade's top, 2^-18 / sqrt(3) = 2.2e-6 in the mean square for the
smallest of a binade and half of that for the largest; queries held so shift a
score of size 1 by as much.  Three terms leave 2^-26; then the fp32 roundings remain:
eight truncated sums of a score and of a tile (2^-24 of their size each, biased),
the exponent's argument and the exponential (2^-24 of up to 8, 2^-22), together a
few 1e-7.  Both are computed below in a model of the arithmetic, on the CPU."""
import math

import numpy as np
import pytest

from tests import branch_util as bu

LIMIT = 2.0 ** -20


# ------------------------------------------------- a model of the arithmetic
def f32(x):
    return np.float32(x).astype(np.float64)


def bf16(x):
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000).astype(np.uint32).view(np.float32).astype(np.float64)


def terms(x, n):
    """x as a sum of n bf16 terms."""
    out, rest = [], f32(x)
    for _ in range(n):
        out.append(bf16(rest))
        rest = f32(rest - out[-1])
    return out


def truncated(x):
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(m * 2.0 ** 24) / 2.0 ** 24, e)


def product(a, b, acc=0.0):
    """acc + a b^T, sixteen inner elements at a time, truncated to fp32 after each."""
    for k in range(0, a.shape[1], 16):
        acc = truncated(acc + a[:, k:k + 16] @ b[:, k:k + 16].T)
    return acc


def model(rng, q, k, v, q_terms=3, w_terms=3, k_terms=1, one_sum=False):
    """The kernels' order of operations; one_sum: the output stays in the tensor cores'
    accumulator over all tiles."""
    c = float(np.float32(1.4426950408889634) / np.float32(math.sqrt(q.shape[1])))
    kt, vt = terms(k, k_terms), terms(v, k_terms)

    def stacked(a, b):  # terms by the size of their products, the smallest added first
        out = 0.0
        for size in reversed(range(max(len(a), len(b)))):
            acc = 0.0
            for i in range(size + 1):
                if i < len(a) and size - i < len(b):
                    acc = product(a[i], b[size - i], acc)
            out = f32(out + acc)
        return out

    s = stacked(terms(q, q_terms), kt)
    base, total, out = np.full((len(q), 1), -1e30), np.zeros((len(q), 1)), np.zeros((len(q), v.shape[1]))
    for t in range(0, len(k), 128):
        x = s[:, t:t + 128]
        top = x.max(1, keepdims=True) * c
        rise = top - base > 8
        new = np.where(rise, f32(top), base)
        corr = f32(np.exp2(np.maximum(base - new, -2000)))
        base, total, out = new, f32(total * corr), f32(out * corr)
        w = f32(np.exp2(f32(x * c - base)) * (1 + rng.uniform(-1, 1, x.shape) * 2.0 ** -22))
        total = f32(total + f32(w.sum(1, keepdims=True)))
        wt, vs = terms(w, w_terms), [y[t:t + 128].T for y in vt]
        out = sum(product(a, vs[0], 0.0) for a in wt[1:]) + product(wt[0], vs[0], out) if one_sum else f32(out + stacked(wt, vs))
    return out / total


def exact(q, k, v):
    s = q @ k.T / math.sqrt(q.shape[1])
    w = np.exp(s - s.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    return w @ v, np.sqrt(w ** 2 @ v ** 2)


def rms(out, want, u):
    return float(np.sqrt((((out - want) / u) ** 2).mean()))


@pytest.mark.parametrize("n,hd", [(9, 128), (9, 64), (139, 128), (2000, 64), (9000, 128)])
@pytest.mark.parametrize("cache_terms", [1, 3])
def test_the_limit_tells_three_terms_from_two(n, hd, cache_terms):
    rng = np.random.default_rng(n + hd)
    q = f32(rng.standard_normal((16, hd)))
    k, v = (f32(rng.standard_normal((n, hd))) for _ in range(2))
    if cache_terms == 1:
        k, v = bf16(k), bf16(v)
    want, u = exact(q, k, v)
    assert rms(model(rng, q, k, v, k_terms=cache_terms), want, u) < LIMIT / 1.5
    assert rms(model(rng, q, k, v, w_terms=2, k_terms=cache_terms), want, u) > LIMIT
    assert rms(model(rng, q, k, v, q_terms=2, k_terms=cache_terms), want, u) > LIMIT
    if cache_terms == 3:
        assert rms(model(rng, q, k, v, k_terms=2), want, u) > LIMIT


def test_the_limit_tells_sums_in_registers_from_sums_in_the_accumulator():
    rng = np.random.default_rng(5)
    q = f32(rng.standard_normal((8, 64)))
    k, v = (bf16(rng.standard_normal((20000, 64))) for _ in range(2))
    v = bf16(v + 1.0)  # (a mean, so that the running sum is large beside what a tile adds)
    want, u = exact(q, k, v)
    assert rms(model(rng, q, k, v, one_sum=True), want, u) > 4 * LIMIT


# ------------------------------------------------------------- the kernels
CASES = [
    # lens, nodes, heads, kv heads, head dim
    ([7, 1, 300], [2, 1, 5], 2, 1, 128), ([131] * 3, [8] * 3, 16, 8, 128), ([9000], [8], 16, 8, 128),
    ([30000], [1], 8, 8, 128), ([9000, 500], [16, 9], 4, 2, 64), ([30000], [32], 2, 1, 128),
    ([9000] * 20, [16] * 20, 2, 1, 128),
    # more than 64 rows to a kv head: few items, shared by clusters, and many
    ([300], [64], 4, 2, 128), ([9000], [64], 4, 2, 64), ([30000], [64], 38, 19, 128), ([2000] * 160, [64] * 160, 2, 1, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["boxes", "rows", "fp32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_tree_attention_holds_24_bits(case, how):
    import torch
    from autoregressive_tts_decode_gb300 import build, q3tts
    build.build()
    lens, nodes, heads, kv_heads, hd = CASES[case]
    page = 12 if how == "rows" else 16
    rng = np.random.default_rng(case)
    dtype = torch.float32 if how == "fp32" else torch.bfloat16
    pool, table = bu.paged_cache(rng, [a + b for a, b in zip(lens, nodes)], page, 1, kv_heads, hd, dtype)
    masks = sum((bu.tree_masks(bu.tree_parents(rng, n)) for n in nodes), [])
    start = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    gen = torch.Generator(device="cuda").manual_seed(case)
    q = torch.randn((len(masks), heads, hd), generator=gen, device="cuda")
    mt = bu.masks_tensor(masks)
    out = q3tts.tree_attention(pool, 0, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                               torch.from_numpy(start).cuda(), mt, q, max_nodes=max(nodes))
    sq = n_el = 0
    for s, (length, n) in enumerate(zip(lens, nodes)):
        pos = torch.arange(length + n, device="cuda")
        kv = pool[0, table[s].long()[pos // page], :, :, pos % page].double()  # [positions, 2, kv heads, hd]
        rows = slice(int(start[s]), int(start[s]) + n)
        bit = (mt[rows, None] >> (pos - length).clamp(0, 63)) & 1
        sees = (pos < length) | (bit != 0)
        for h in range(heads):
            k, v = kv[:, 0, h // (heads // kv_heads)], kv[:, 1, h // (heads // kv_heads)]
            w = torch.softmax((q[rows, h].double() @ k.T / math.sqrt(hd)).masked_fill(~sees, -math.inf), -1)
            off = (out[rows, h].double() - w @ v) / (w ** 2 @ v ** 2).sqrt()
            sq += float((off ** 2).sum())
            n_el += off.numel()
    assert math.sqrt(sq / n_el) < LIMIT, math.sqrt(sq / n_el) / LIMIT
