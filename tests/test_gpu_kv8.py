"""The 8-bit cache's operators on the GPU against their definitions in 64 bits:
quantising writes, reading back, attention, and a stream that uses them together."""
import math

import numpy as np
import pytest

from tests import branch_util as bu
from tests import kv8_util as ku

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from autoregressive_tts_decode_gb300 import build, q3tts
    build.build()
    return q3tts


def dt(name):
    import torch
    return getattr(torch, name)


def randn(rng, shape, dtype):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 31)))
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def same_values(codes, want):
    """codes: float8 tensor; want: float64 numpy (NaN where the code is NaN)."""
    got = ku.VALUES[codes.view(dt("uint8")).cpu().numpy()]
    return bool(np.array_equal(got, want, equal_nan=True))


# ------------------------------------------------------------------ write
WRITES = [
    # lens, rows, kv heads, head dim, page, block
    ([0], [1], 1, 128, 16, 16), ([131], [1], 8, 128, 16, 16), ([0, 5, 16, 31], [1, 1, 1, 1], 2, 64, 16, 16),
    ([0, 3, 15, 16, 17], [1, 40, 1, 16, 33], 2, 128, 16, 16), ([7, 0, 100], [0, 0, 5], 3, 64, 12, 4),
    ([5], [70], 2, 128, 64, 64), ([9, 1], [130, 3], 1, 64, 24, 24), ([3, 0], [20, 9], 2, 128, 16, 1),
    ([250, 1], [300, 2], 2, 128, 32, 8), ([11], [37], 5, 64, 8, 2), ([0], [200], 1, 128, 128, 128),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("case", WRITES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_write(q3, case, dtype):
    """Codes and powers are exactly the definition's; what is not written stays. Rows
    come with the pitch of a projection's output, and their sizes span many powers."""
    import torch
    lens, rows, kvh, hd, page, block = case
    rng = np.random.default_rng(1)
    total = [a + b for a, b in zip(lens, rows)]
    codes, powers, table = ku.cache(rng, total, page, block, 2, kvh, hd, 110, 125)
    n = sum(rows)
    qkv = randn(rng, (n, 3 * kvh, hd), torch.float32) * torch.exp2(randn(rng, (n, 3 * kvh, 1), torch.float32) * 4)
    qkv = qkv.to(dt(dtype))
    k, v = qkv[:, kvh:2 * kvh], qkv[:, 2 * kvh:]
    want, wpow = ku.write_reference(codes, powers, 1, table, lens, rows, k.double().cpu().numpy(), v.double().cpu().numpy())
    pool, scales, tab = ku.to_gpu(codes, powers, table)
    status = ku.ints([0])
    q3.kv8_write(pool, scales, 1, tab, ku.ints(lens), ku.ints(ku.starts(rows)), k, v, max_rows=max(rows), status=status)
    assert int(status) == 0
    assert np.array_equal(scales.view(torch.uint8).cpu().numpy(), wpow) and same_values(pool, want)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_write_of_extremes(q3, dtype):
    """Magnitudes at the borders of powers, the type's largest and smallest, zeroes,
    infinities and NaN, in fresh blocks and behind rows that are there."""
    import torch
    t = dt(dtype)
    big, tiny = float(torch.finfo(t).max), float(torch.finfo(t).smallest_normal)
    tops = [448.0, 448.0 * (1 + torch.finfo(t).eps), 449.0, 480.0, 512.0, 1.75, 1.76, 0.0, big, tiny, tiny / 2 ** 5, math.inf,
            math.nan, 2.0 ** -100]
    rng = np.random.default_rng(2)
    lens, rows = [0, 3] * len(tops), [2, 2] * len(tops)
    codes, powers, table = ku.cache(rng, [5] * len(lens), 16, 8, 1, 1, 64, 100, 140)
    x = (randn(rng, (2 * len(lens), 1, 64), torch.float32).clamp(-1, 1)).to(t)
    for i in range(len(lens)):
        top = tops[i // 2]
        if math.isfinite(top):
            x[2 * i:2 * i + 2] = (x[2 * i:2 * i + 2].double() * top).to(t)
        x[2 * i, 0, 17] = top
        x[2 * i + 1, 0, 3] = -top
        x[2 * i, 0, 5] = math.nan if i % 3 == 0 else -math.inf if i % 3 == 1 else 0.0
    kk = x.double().cpu().numpy()
    want, wpow = ku.write_reference(codes, powers, 0, table, lens, rows, kk, kk)
    pool, scales, tab = ku.to_gpu(codes, powers, table)
    q3.kv8_write(pool, scales, 0, tab, ku.ints(lens), ku.ints(ku.starts(rows)), x, x)
    assert np.array_equal(scales.view(torch.uint8).cpu().numpy(), wpow) and same_values(pool, want)


def test_write_row_by_row_is_a_blocks_write_rounded_again(q3):
    """A block that is filled a position at a time: the power is the whole block's, and
    each code is within a rounding of the larger powers of the value."""
    import torch
    rng = np.random.default_rng(3)
    hd, rows = 128, 16
    x = randn(rng, (rows, 1, hd), torch.float32) * torch.exp2(randn(rng, (rows, 1, 1), torch.float32) * 2)
    codes, powers, table = ku.cache(rng, [0], 16, 16, 1, 1, hd)
    pool, scales, tab = ku.to_gpu(np.concatenate([codes] * 2, 1), np.concatenate([powers] * 2, 1), np.zeros_like(table))
    for i in range(rows):
        q3.kv8_write(pool, scales, 0, tab, ku.ints([i]), ku.ints([0, 1]), x[i:i + 1], x[i:i + 1])
    q3.kv8_write(pool, scales, 0, tab + 1, ku.ints([0]), ku.ints([0, rows]), x, x)
    p = scales.view(torch.uint8)
    assert torch.equal(p[0, 0], p[0, 1])
    two = 2.0 ** (int(p[0, 0, 0, 0, 0]) - 127)
    a, b = (pool[0, i, 0, 0].float().double() * two for i in (0, 1))
    want = x[:, 0].double()
    half = torch.maximum(want.abs() * 2.0 ** -4, torch.full_like(want, 2.0 ** -10 * two))
    assert bool(((b - want).abs() <= half).all())
    # a code was rounded once for each of the powers it was held at, the earlier ones at finer steps
    ups = len({int(v) for v in [ku.power(float(x[:i + 1].abs().max())) for i in range(rows)]})
    assert bool(((a - want).abs() <= ups * 1.0625 * half).all())


def test_write_leaves_out_what_does_not_fit(q3):
    """Lengths, rows and page ids that do not fit: reported, nothing of them written."""
    import torch
    rng = np.random.default_rng(4)
    lens, rows = [3, 20, 5, 4], [4, 4, 4, 4]
    codes, powers, table = ku.cache(rng, [40] * 4, 16, 8, 1, 2, 64)
    k = randn(rng, (16, 2, 64), torch.float32)
    kk = k.double().cpu().numpy()

    def run(lens_, start_, table_, most=4):
        pool, scales, _ = ku.to_gpu(codes, powers, table)
        status = ku.ints([0])
        q3.kv8_write(pool, scales, 0, ku.ints(table_), ku.ints(lens_), ku.ints(start_), k, k, max_rows=most, status=status)
        return pool, scales, int(status)

    ok, okp = ku.write_reference(codes, powers, 0, table, lens, rows, kk, kk)
    start = ku.starts(rows)
    for change in ("length", "negative", "most", "page", "negative page", "start"):
        ln, st, tb, most = list(lens), start.copy(), table.copy(), 4
        keep = [0, 1, 2, 3]
        if change == "length":
            ln[1] = 16 * table.shape[1] - 3
            keep = [0, 2, 3]
        elif change == "negative":
            ln[2] = -1
            keep = [0, 1, 3]
        elif change == "most":
            st = np.array([0, 5, 8, 12, 16], np.int32)
            keep = None
        elif change == "page":
            tb[1, 1] = codes.shape[1]
            keep = [0, 2, 3]
        elif change == "negative page":
            tb[3, 0] = -1
            keep = [0, 1, 2]
        else:
            st = np.array([0, 4, 8, 12, 17], np.int32)
            keep = [0, 1, 2]
        pool, scales, code = run(ln, st, tb, most)
        assert code == q3.ERR_ARG, change
        if keep is None:
            continue
        want, wpow = ku.VALUES[codes].copy(), powers.copy()
        for s in keep:
            for j in range(table.shape[1]):
                if table[s, j] < codes.shape[1]:
                    want[:, table[s, j]], wpow[:, table[s, j]] = ok[:, table[s, j]], okp[:, table[s, j]]
        assert np.array_equal(scales.view(torch.uint8).cpu().numpy(), wpow) and same_values(pool, want), change


# ------------------------------------------------------------------- read
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("path", [False, True])
@pytest.mark.parametrize("lens,rows,kvh,hd,page,block", [
    ([0], [1], 1, 128, 16, 16), ([131, 0, 7], [4, 60, 0], 8, 128, 16, 16), ([5, 0], [33, 16], 3, 64, 12, 4),
    ([100], [300], 2, 128, 64, 1), ([0, 1, 2], [17, 31, 100], 2, 64, 8, 8)])
def test_read(q3, lens, rows, kvh, hd, page, block, path, dtype):
    import torch
    t = dt(dtype)
    rng = np.random.default_rng(5)
    codes, powers, table = ku.cache(rng, [a + b for a, b in zip(lens, rows)], page, block, 2, kvh, hd, 0, 247)
    pool, scales, tab = ku.to_gpu(codes, powers, table)
    n, start = sum(rows), ku.starts(rows)
    offs = [rng.integers(0, r, r) if path else np.arange(r) for r in rows]
    buf = torch.full((n + 2, 3 * kvh, hd), -7.5, dtype=t, device="cuda")  # interleaved, rows before and behind
    out = buf[:, :kvh], buf[:, 2 * kvh:]
    p = ku.ints(np.concatenate([[0], *offs, [0]])) if path else None
    got = q3.kv8_read(pool, scales, 1, tab, ku.ints(lens), ku.ints(start + 1), path=p, max_rows=max(rows), out=out)
    assert got is out
    want = buf.clone().fill_(-7.5)
    for s, length in enumerate(lens):
        c, w = ku.values(codes, powers, 1, table, s, length + offs[s])
        for j, at in enumerate((0, 2 * kvh)):
            x = torch.from_numpy(c[j] * w[j][..., None]).cuda()
            # (through fp32, where these are exact, so that bf16 is rounded once)
            want[1 + start[s]:1 + start[s + 1], at:at + kvh] = x.float().to(t)
    assert torch.equal(buf, want)


def test_read_leaves_out_what_does_not_fit(q3):
    import torch
    rng = np.random.default_rng(6)
    codes, powers, table = ku.cache(rng, [20, 20], 16, 16, 1, 1, 64)
    pool, scales, tab = ku.to_gpu(codes, powers, table)
    start, path = ku.ints([0, 3, 6]), [0, 1, 2, 0, 1, 2]
    good = q3.kv8_read(pool, scales, 0, tab, ku.ints([4, 4]), start, path=ku.ints(path))
    for at, bad in ((1, -1), (4, 16 * table.shape[1]), (2, 1 << 30)):
        p = list(path)
        p[at] = bad
        status, out = ku.ints([0]), tuple(torch.full_like(g, 9.0) for g in good)
        q3.kv8_read(pool, scales, 0, tab, ku.ints([4, 4]), start, path=ku.ints(p), out=out, status=status)
        assert int(status) == q3.ERR_ARG
        for o, g in zip(out, good):
            keep = [i for i in range(6) if i != at]
            assert torch.equal(o[keep], g[keep]) and bool((o[at] == 9.0).all())
    bad = tab.clone()
    bad[1, 0] = pool.shape[1]
    status, out = ku.ints([0]), tuple(torch.full_like(g, 9.0) for g in good)
    q3.kv8_read(pool, scales, 0, bad, ku.ints([4, 4]), start, path=ku.ints(path), out=out, status=status)
    assert int(status) == q3.ERR_ARG
    for o, g in zip(out, good):
        assert torch.equal(o[:3], g[:3]) and bool((o[3:] == 9.0).all())


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_rows_that_are_not_aligned(q3, dtype):
    """Rows at odd addresses with odd pitches, read and written: as aligned ones."""
    import torch
    rng, t = np.random.default_rng(24), dt(dtype)
    lens, rows, kvh, hd = [3, 20, 0], [40, 1, 18], 3, 64
    codes, powers, table = ku.cache(rng, [a + b for a, b in zip(lens, rows)], 16, 8, 1, kvh, hd)
    n, start = sum(rows), ku.ints(ku.starts(rows))
    pitch = 2 * kvh * hd + 1
    kv = torch.empty(n * pitch + 3, dtype=t, device="cuda")[3:].view(n, pitch)
    k, v = (kv[:, i * kvh * hd:(i + 1) * kvh * hd].unflatten(1, (kvh, hd)) for i in (0, 1))
    k.copy_(randn(rng, (n, kvh, hd), t))
    v.copy_(randn(rng, (n, kvh, hd), t))
    got = []
    for a, b in ((k, v), (k.contiguous(), v.contiguous())):
        pool, scales, tab = ku.to_gpu(codes, powers, table)
        q3.kv8_write(pool, scales, 0, tab, ku.ints(lens), start, a, b)
        got.append((pool.view(torch.uint8), scales.view(torch.uint8)))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    kv.fill_(-7.5)
    want = q3.kv8_read(pool, scales, 0, tab, ku.ints(lens), start, out=(torch.empty((n, kvh, hd), dtype=t, device="cuda"),
                                                                        torch.empty((n, kvh, hd), dtype=t, device="cuda")))
    q3.kv8_read(pool, scales, 0, tab, ku.ints(lens), start, out=(k, v))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and bool((kv[:, -1] == -7.5).all())


def test_offsets_past_32_bits(q3):
    """A cache of 9 GB whose used pages are its last ones: as one that has no others."""
    import torch
    rng = np.random.default_rng(25)
    lens, rows, kvh, hd, page = [200, 0], [90, 1], 8, 128, 16
    codes, powers, table = ku.cache(rng, [a + b for a, b in zip(lens, rows)], page, 16, 1, kvh, hd)
    small, sp, tab = ku.to_gpu(codes, powers, table)
    pages = codes.shape[1]
    before = 9 * (1 << 30) // (2 * kvh * page * hd) - pages
    big = torch.empty((1, before + pages, 2, kvh, page, hd), dtype=torch.uint8, device="cuda")
    bp = torch.empty((1, before + pages, 2, kvh, 1), dtype=torch.uint8, device="cuda")
    big[:, before:] = small.view(torch.uint8)
    bp[:, before:] = sp.view(torch.uint8)
    moved = torch.where(tab < pages, tab + before, tab)
    start, ln = ku.ints(ku.starts(rows)), ku.ints(lens)
    k, v, q = (randn(rng, (91, h, hd), torch.bfloat16) for h in (kvh, kvh, 16))
    results = []
    for pool, scales, t in ((small, sp, tab), (big.view(torch.float8_e4m3fn), bp.view(torch.float8_e8m0fnu), moved)):
        q3.kv8_write(pool, scales, 0, t, ln, start, k, v, max_rows=90)
        few = q3.kv8_attention(pool, scales, 0, t, ku.ints([289, 0]), ku.ints([0, 1, 2]), q[:2].contiguous(), max_rows=1)
        results.append((q3.kv8_attention(pool, scales, 0, t, ln, start, q, max_rows=90), few,
                        *q3.kv8_read(pool, scales, 0, t, ln, start, path=ku.ints([*range(90), 0]), max_rows=90)))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert torch.equal(big[:, before:], small.view(torch.uint8)) and torch.equal(bp[:, before:], sp.view(torch.uint8))


def test_a_power_of_255_reads_as_nan(q3):
    import torch
    codes, powers, table = ku.cache(np.random.default_rng(7), [4], 16, 16, 1, 1, 64)
    powers[:] = 255
    pool, scales, tab = ku.to_gpu(codes, powers, table)
    k, v = q3.kv8_read(pool, scales, 0, tab, ku.ints([0]), ku.ints([0, 4]), path=ku.ints([0, 1, 2, 3]))
    assert bool(torch.isnan(k).all()) and bool(torch.isnan(v).all())


# -------------------------------------------------------------- attention
def attend_case(rng, lens, rows, heads, kvh, hd, page, block, dtype, tree, layers=2, lo=121, hi=130):
    import torch
    codes, powers, table = ku.cache(rng, [a + b for a, b in zip(lens, rows)], page, block, layers, kvh, hd, lo, hi)
    masks = None
    if tree:
        masks = []
        for n in rows:
            masks += bu.tree_masks(bu.tree_parents(rng, n))
    q = randn(rng, (sum(rows), heads, hd), dt(dtype))
    # codes are of size 100 or so, powers of 1: scores of a few units
    q = (q.float() * 2.0 ** -8).to(q.dtype)
    return dict(codes=codes, powers=powers, table=table, lens=lens, rows=rows, masks=masks, q=q)


def run_attention(q3, c, layer=1, **kw):
    pool, scales, tab = ku.to_gpu(c["codes"], c["powers"], c["table"])
    m = None if c["masks"] is None else bu.masks_tensor(c["masks"])
    return q3.kv8_attention(pool, scales, layer, tab, ku.ints(c["lens"]), ku.ints(ku.starts(c["rows"])), c["q"], masks=m,
                            max_rows=max(1, max(c["rows"])), **kw)


def check_attention(c, out, layer=1):
    want, tol = ku.attention_reference(c["codes"], c["powers"], layer, c["table"], c["lens"], c["rows"], c["masks"], c["q"])
    off = (out.double() - want).abs() / tol
    assert bool((off <= 1).all()), f"{float(off.max()):.3g} of the bound"


TREES = [
    # lens, rows, heads, kv heads, head dim, page, block
    ([0], [1], 2, 1, 64, 16, 16), ([1], [1], 4, 2, 128, 16, 16), ([0], [64], 2, 1, 128, 16, 16),
    ([131], [8], 16, 8, 128, 16, 16), ([127, 128, 129], [1, 1, 1], 4, 2, 128, 16, 8),
    ([15, 16, 17, 0], [1, 16, 17, 3], 4, 2, 64, 16, 4), ([100, 0, 50], [0, 5, 0], 4, 2, 128, 16, 16),
    ([777, 3, 260], [64, 1, 33], 8, 2, 128, 16, 1), ([500], [9], 3, 3, 64, 12, 4), ([200, 31], [7, 2], 8, 1, 128, 8, 8),
    ([300], [20], 12, 3, 128, 32, 32), ([129], [5], 4, 2, 64, 64, 16), ([511], [40], 4, 4, 64, 128, 64),
    ([600], [13], 4, 2, 128, 256, 128), ([70], [64], 16, 1, 64, 16, 16), ([45], [6], 2, 1, 128, 1, 1),
    ([2048], [16], 16, 8, 128, 16, 16), ([5000, 1], [3, 3], 2, 1, 64, 16, 16), ([333], [17], 10, 2, 128, 24, 12),
    ([9000], [64], 4, 2, 128, 16, 16), ([960, 3, 0], [64, 33, 40], 16, 2, 128, 16, 2), ([383], [22], 3, 1, 64, 256, 256),
    ([127, 64, 0, 200] * 5, [64, 64, 64, 10] * 5, 4, 2, 128, 8, 8), ([500, 129] * 4, [64, 50] * 4, 8, 2, 64, 32, 8),
    ([90], [2], 1024, 1, 64, 16, 16), ([40, 0, 200], [33, 1, 16], 14, 2, 64, 12, 12), ([37], [5], 999, 1, 128, 4, 4),
]
CHUNKS = [
    ([0], [1], 4, 2, 128, 16, 16), ([0], [130], 4, 2, 128, 16, 16), ([0], [1982], 4, 2, 128, 16, 16),
    ([0, 37, 5], [200, 1, 129], 4, 2, 128, 16, 16), ([1000], [300], 2, 1, 64, 16, 16), ([128], [128], 8, 4, 128, 32, 8),
    ([61], [190], 6, 2, 64, 12, 4), ([777, 0], [65, 257], 16, 2, 128, 64, 64), ([5], [70], 32, 1, 64, 24, 24),
    ([3000], [500], 2, 2, 128, 128, 32), ([0, 9, 200, 1] * 6, [1, 128, 64, 90] * 6, 4, 2, 64, 8, 1),
    ([1, 1000, 131, 0] * 3, [1] * 12, 16, 8, 128, 16, 16), ([5000], [1], 2, 1, 64, 256, 256), ([20000], [1], 4, 1, 128, 16, 16),
    ([16383], [1], 8, 8, 128, 16, 16), ([700, 31], [1, 1], 5, 5, 64, 16, 8), ([64], [3], 300, 2, 128, 16, 16),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("tree,case", [(True, c) for c in TREES] + [(False, c) for c in CHUNKS],
                         ids=lambda c: "-".join(str(x) for x in c).replace(" ", "")[:60] if isinstance(c, tuple) else str(c))
def test_attention(q3, case, tree, dtype):
    c = attend_case(np.random.default_rng(8), *case, dtype=dtype, tree=tree)
    status = ku.ints([0])
    out = run_attention(q3, c, status=status)
    assert out.dtype == c["q"].dtype
    check_attention(c, out)
    assert int(status) == 0


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("tree,seqs,longest,most,heads,kvh,hd,page,block", [
    (True, 97, 700, 13, 16, 8, 128, 16, 16), (True, 60, 1500, 1, 8, 8, 128, 16, 16), (True, 300, 90, 3, 4, 2, 64, 16, 8),
    (True, 45, 600, 40, 8, 4, 128, 16, 16), (True, 33, 800, 64, 2, 1, 64, 24, 8), (False, 41, 900, 1, 16, 8, 128, 12, 12),
    (False, 60, 300, 100, 8, 4, 128, 16, 16), (False, 170, 300, 33, 8, 1, 64, 64, 16), (False, 300, 40, 1, 4, 4, 128, 8, 4),
    (False, 270, 60, 40, 8, 1, 64, 16, 8), (True, 300, 150, 30, 8, 1, 128, 5, 5), (False, 70, 500, 60, 12, 3, 128, 200, 8)])
def test_attention_of_many_sequences(q3, dtype, tree, seqs, longest, most, heads, kvh, hd, page, block):
    import torch
    rng = np.random.default_rng(9)
    lens, rows = rng.integers(0, longest, seqs).tolist(), rng.integers(0, most + 1, seqs).tolist()
    c = attend_case(rng, lens, rows, heads, kvh, hd, page, block, dtype, tree)
    status = ku.ints([0])
    out = run_attention(q3, c, status=status)
    check_attention(c, out)
    assert int(status) == 0 and torch.equal(out, run_attention(q3, c))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("case", [([61, 0], [90, 33], 4, 2, 64, 1, 1), ([300], [70], 4, 2, 128, 3, 1), ([131], [100], 6, 2, 128, 5, 5),
                                  ([450, 7], [80, 1], 4, 2, 128, 200, 8), ([450, 130], [1, 1], 4, 2, 64, 200, 40), ([700], [120], 2, 1, 64, 384, 96),
                                  ([255, 256, 257], [65, 64, 63], 2, 1, 128, 128, 2)])
def test_attention_over_pages_of_all_sizes(q3, case, dtype):
    """Pages of one position, of odd numbers, larger than a tile and no multiple of it; the most
    rows of a sequence left to the default."""
    import torch
    c = attend_case(np.random.default_rng(23), *case, dtype=dtype, tree=False)
    pool, scales, tab = ku.to_gpu(c["codes"], c["powers"], c["table"])
    out = q3.kv8_attention(pool, scales, 1, tab, ku.ints(c["lens"]), ku.ints(ku.starts(c["rows"])), c["q"])
    check_attention(c, out)
    assert torch.equal(out, run_attention(q3, c)) or max(c["rows"]) != sum(c["rows"])


# rows, heads, kv heads, positions, sequences; the last three fill the GPU with tiles of 128 rows
SHAPES = [(1, 4, 2, 300, 1), (13, 4, 2, 300, 1), (64, 4, 2, 500, 1), (40, 16, 1, 77, 1), (1, 2, 1, 3000, 1), (5, 8, 1, 129, 1),
          (64, 4, 2, 200, 60), (33, 16, 2, 77, 50), (20, 8, 1, 300, 110)]


@pytest.mark.parametrize("rows,heads,kvh,length,seqs", SHAPES)
@pytest.mark.parametrize("tree", [True, False])
def test_attention_over_blocks_of_all_sizes(q3, tree, rows, heads, kvh, length, seqs):
    """Powers from 2^-40 to 2^40 in one sequence (queries small, so that scores stay in
    their range): small values count where the large ones get no weight."""
    c = attend_case(np.random.default_rng(10), [length] * seqs, [rows] * seqs, heads, kvh, 128, 16, 4, "float32", tree, lo=87, hi=167)
    c["powers"][:, :, 0] = np.where(c["powers"][:, :, 0] == 255, 255, 120)
    check_attention(c, run_attention(q3, c))


@pytest.mark.parametrize("rows,heads,kvh,length,seqs", SHAPES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_scores_far_apart(q3, rows, heads, kvh, length, seqs, dtype):
    """Scores up to hundreds: the largest rises from tile to tile, nearly all weights vanish."""
    c = attend_case(np.random.default_rng(11), [length] * seqs, [rows] * seqs, heads, kvh, 128, 16, 16, dtype, False)
    c["q"] = (c["q"].float() * 16).to(c["q"].dtype)
    check_attention(c, run_attention(q3, c))


@pytest.mark.parametrize("rows,heads,kvh,length,seqs", SHAPES)
def test_rows_that_see_nothing_and_rows_that_do_not_see_nan(q3, rows, heads, kvh, length, seqs):
    """Masks of nothing (over an empty context: zeroes), and nodes that are NaN or huge, in
    their codes and in their blocks' powers, seen by none of the others."""
    import torch
    rng, n = np.random.default_rng(12), seqs + 1
    for ctx in (0, length):
        c = attend_case(rng, [ctx] * n, [rows] * n, heads, kvh, 64, 16, 1, "float32", True)
        c["masks"] = [m & ~1 if i % rows else 0 for i, m in enumerate(c["masks"])]
        if rows > 2:  # none sees node 1 either
            c["masks"] = [m & ~2 for m in c["masks"]]
        for s in range(n):
            for node, power in ((0, 255), (1, 254)):
                if node < rows:
                    pos = ctx + node
                    pg, slot = c["table"][s, pos // 16], pos % 16
                    if node == 0:
                        c["codes"][:, pg, :, :, slot] = ku.NAN
                    c["powers"][:, pg, :, :, slot] = power if node == 0 or rows > 2 else 127
        out = run_attention(q3, c)
        check_attention(c, out)
        if ctx == 0:
            assert bool((out[::rows] == 0).all())


@pytest.mark.parametrize("seqs", [1, 60])
@pytest.mark.parametrize("rows", [1, 40, 64])
def test_a_row_that_sees_nan_is_nan_alone(q3, rows, seqs):
    """A NaN value that one node of each sequence sees: its row is NaN, the others' results
    do not change."""
    import torch
    c = attend_case(np.random.default_rng(13), [200] * seqs, [rows] * seqs, 4, 2, 128, 16, 16, "float32", True)
    want = run_attention(q3, c)
    pos = 200 + rows - 1
    for s in range(seqs):
        c["codes"][:, c["table"][s, pos // 16], 1, :, pos % 16, 7] = ku.NAN
    out = run_attention(q3, c)
    last = torch.arange(rows * seqs, device="cuda") % rows == rows - 1
    assert torch.equal(out[~last], want[~last]) and bool(torch.isnan(out[last, :, 7]).all())


@pytest.mark.parametrize("rows,heads,kvh,length,seqs", SHAPES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_pitches_and_rows_outside_the_sequences(q3, rows, heads, kvh, length, seqs, dtype):
    """Queries and outputs inside wider rows, at addresses that are not multiples of 16
    bytes; rows before the first sequence and behind the last are left alone."""
    import torch
    hd, extra = 64, 1
    c = attend_case(np.random.default_rng(14), [length] * seqs + [3], [rows] * seqs + [1], heads, kvh, hd, 16, 16, dtype, False)
    want = run_attention(q3, c)
    n = rows * seqs + 1
    buf = torch.full(((n + 4) * (heads * hd + extra) + 9,), -7.5, dtype=c["q"].dtype, device="cuda")

    def view():
        return buf.clone()[3:3 + (n + 4) * (heads * hd + extra)].view(n + 4, -1)[:, :heads * hd].unflatten(1, (heads, hd))

    q, out = view(), view()
    q[2:-2] = c["q"]
    pool, scales, tab = ku.to_gpu(c["codes"], c["powers"], c["table"])
    q3.kv8_attention(pool, scales, 1, tab, ku.ints(c["lens"]), ku.ints(ku.starts(c["rows"]) + 2), q, max_rows=rows, out=out)
    assert torch.equal(out[2:-2], want) and bool((out[:2] == -7.5).all()) and bool((out[-2:] == -7.5).all())


@pytest.mark.parametrize("rows,seqs", [(1, 3), (3, 3), (50, 3), (50, 70)])
@pytest.mark.parametrize("tree", [True, False])
def test_attention_leaves_out_what_does_not_fit(q3, rows, seqs, tree):
    import torch
    lens = ([100, 200, 150] * seqs)[:seqs]
    c = attend_case(np.random.default_rng(15), lens, [rows] * seqs, 4, 2, 128, 16, 16, "float32", tree)
    want = run_attention(q3, c)
    cap = 16 * c["table"].shape[1]
    for bad in (cap - rows + 1, -1, 1 << 30):
        d = dict(c, lens=[100, bad, *lens[2:]])
        out, status = torch.full_like(want, 3.0), ku.ints([0])
        run_attention(q3, d, out=out, status=status)
        assert int(status) == q3.ERR_ARG
        assert torch.equal(out[:rows], want[:rows]) and torch.equal(out[2 * rows:], want[2 * rows:])
        assert bool((out[rows:2 * rows] == 3.0).all())
    table = c["table"].copy()
    table[1, 2] = -5
    status = ku.ints([0])
    out = run_attention(q3, dict(c, table=table), status=status)
    assert int(status) == q3.ERR_ARG
    assert torch.equal(out[:rows], want[:rows]) and torch.equal(out[2 * rows:], want[2 * rows:])


# --------------------------------------------------------------- together
def test_a_stream_over_the_cache(q3):
    """A prompt in two chunks, single tokens, a drafted tree whose accepted path moves up:
    each attention is that of the rows that were written, at the cache's own rounding."""
    import torch
    rng = np.random.default_rng(16)
    kvh, heads, hd, page, block = 2, 4, 128, 16, 16
    codes, powers, table = ku.cache(rng, [400, 400], page, block, 2, kvh, hd)
    pool, scales, tab = ku.to_gpu(np.full_like(codes, ku.NAN), np.full_like(powers, 255), table)
    lens = [0, 0]
    held = [torch.zeros((0, 2, kvh, hd), dtype=torch.float64, device="cuda") for _ in range(2)]

    def host():
        return pool.view(torch.uint8).cpu().numpy(), scales.view(torch.uint8).cpu().numpy()

    def step(rows, masks=None):
        n = sum(rows)
        k, v, q = (randn(rng, (n, h, hd), torch.bfloat16) for h in (kvh, kvh, heads))
        start = ku.ints(ku.starts(rows))
        q3.kv8_write(pool, scales, 1, tab, ku.ints(lens), start, k, v, max_rows=max(rows))
        m = None if masks is None else bu.masks_tensor(masks)
        out = q3.kv8_attention(pool, scales, 1, tab, ku.ints(lens), start, q, masks=m, max_rows=max(rows))
        c, p = host()
        want, tol = ku.attention_reference(c, p, 1, table, lens, rows, masks, q)
        assert bool(((out.double() - want).abs() <= tol).all())
        return torch.stack([k, v], 1).double()

    def keep(rows, kv, at=None):
        r0 = 0
        for s, n in enumerate(rows):
            held[s] = torch.cat([held[s], kv[r0:r0 + n] if at is None else kv[r0:r0 + n][at[s]]])
            lens[s] = len(held[s])
            r0 += n

    for rows in ([100, 37], [70, 120], [1, 1], [1, 1], [1, 1]):
        keep(rows, step(rows))
    rows = [9, 17]
    parents = [bu.tree_parents(rng, n) for n in rows]
    kv = step(rows, [m for p in parents for m in bu.tree_masks(p)])
    path = []
    for p in parents:  # the last node and its ancestors
        at, line = len(p) - 1, []
        while at >= 0:
            line.append(at)
            at = p[at]
        path.append(line[::-1])
    start = ku.ints(ku.starts([len(p) for p in path]))
    got = q3.kv8_read(pool, scales, 1, tab, ku.ints(lens), start, path=ku.ints(np.concatenate(path)))
    q3.kv8_write(pool, scales, 1, tab, ku.ints(lens), start, *got)
    keep(rows, kv, path)
    keep([1, 1], step([1, 1]))
    # what the cache holds is what was written, to a rounding at each power (three at most moved it)
    for s in range(2):
        c, p = ku.values(*host(), 1, table, s, np.arange(lens[s]))
        for j in range(2):
            x = torch.from_numpy(c[j] * p[j][..., None]).cuda()
            step_ = torch.from_numpy(p[j][..., None] * 2.0 ** -10).cuda()
            want = held[s][:, j]
            assert bool(((x - want).abs() <= 4 * torch.maximum(want.abs() * 2.0 ** -4, step_.expand_as(want))).all())


def test_captured_on_another_stream(q3):
    """Write, attention and read in a graph on a side stream, replayed on new rows; two
    calls at once on two streams do not meet."""
    import torch
    c = attend_case(np.random.default_rng(17), [130, 700], [1, 1], 16, 8, 128, 16, 16, "bfloat16", False)
    pool, scales, tab = ku.to_gpu(c["codes"], c["powers"], c["table"])
    lens, start = ku.ints(c["lens"]), ku.ints([0, 1, 2])
    k, v, q = (randn(np.random.default_rng(18), (2, h, 128), torch.bfloat16) for h in (8, 8, 16))
    out, back = torch.empty_like(q), (torch.empty_like(k), torch.empty_like(v))

    def calls():
        q3.kv8_write(pool, scales, 1, tab, lens, start, k, v, max_rows=1)
        q3.kv8_attention(pool, scales, 1, tab, lens, start, q, max_rows=1, out=out)
        q3.kv8_read(pool, scales, 1, tab, lens, start, max_rows=1, out=back)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls()
    for seed in (19, 20):
        rng = np.random.default_rng(seed)
        for t, h in ((k, 8), (v, 8), (q, 16)):
            t.copy_(randn(rng, (2, h, 128), torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), back[0].clone(), back[1].clone()
        pool2, scales2, _ = ku.to_gpu(c["codes"], c["powers"], c["table"])
        pool2.view(torch.uint8).copy_(pool.view(torch.uint8))
        scales2.view(torch.uint8).copy_(scales.view(torch.uint8))
        want = q3.kv8_attention(pool2, scales2, 1, tab, lens, start, q, max_rows=1)
        b2 = q3.kv8_read(pool2, scales2, 1, tab, lens, start, path=ku.ints([0, 0]))
        assert torch.equal(got[0], want) and torch.equal(got[1], b2[0]) and torch.equal(got[2], b2[1])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                outs.append(q3.kv8_attention(pool, scales, 1, tab, lens, start, q, max_rows=1))
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_binding_refuses(q3):
    """Wrong shapes, types, devices and strides are errors before any launch."""
    import torch
    c = attend_case(np.random.default_rng(21), [20], [2], 4, 2, 64, 16, 8, "float32", True)
    pool, scales, tab = ku.to_gpu(c["codes"], c["powers"], c["table"])
    lens, start = ku.ints([20]), ku.ints([0, 2])
    k = torch.zeros((2, 2, 64), device="cuda")
    m = bu.masks_tensor(c["masks"])
    good = dict(pool=pool, scales=scales, layer=0, page_table=tab, lengths=lens, start=start)
    bad = [dict(pool=pool.cpu()), dict(pool=pool.view(torch.uint8)), dict(pool=pool[..., :32]), dict(pool=pool[:, :, :1]),
           dict(scales=scales[..., :1]), dict(scales=scales.float()), dict(scales=scales.view(torch.uint8).cpu()),
           dict(layer=2), dict(page_table=tab[0]), dict(page_table=tab.long()), dict(lengths=ku.ints([20, 3])),
           dict(lengths=lens.cpu()), dict(start=ku.ints([0]))]
    calls = [lambda a, **kw: q3.kv8_write(**a, **{**dict(k=k, v=k), **kw}),
             lambda a, **kw: q3.kv8_read(**a, **{**dict(path=ku.ints([0, 1])), **kw}),
             lambda a, **kw: q3.kv8_attention(**a, **{**dict(q=c["q"], masks=m), **kw})]
    for call in calls:
        call(good)
        for b in bad:
            with pytest.raises(q3.Q3TTSError):
                call({**good, **b})
        for kw in (dict(max_rows=0), dict(status=torch.zeros(1, device="cuda")), dict(status=ku.ints([0, 0]))):
            with pytest.raises(q3.Q3TTSError):
                call(good, **kw)
    for kw in (dict(k=k.half()), dict(v=k.bfloat16()), dict(k=k.transpose(0, 1)), dict(v=k[:1]), dict(k=k.cpu()),
               dict(k=k[..., ::2])):
        with pytest.raises(q3.Q3TTSError):
            calls[0](good, **kw)
    for kw in (dict(path=None), dict(path=ku.ints([0]), out=(k, k.clone())), dict(out=(k, k)),
               dict(out=(k, k.bfloat16())), dict(path=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(q3.Q3TTSError):
            calls[1](good, **kw)
    q = c["q"]
    for kw in (dict(q=q[:, :3]), dict(q=q.half()), dict(out=q), dict(out=q.bfloat16()), dict(masks=m[:1]),
               dict(masks=m.int()), dict(max_rows=65), dict(q=q[..., :32])):
        with pytest.raises(q3.Q3TTSError):
            calls[2](good, **kw)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("case,tile", [(([300], [1], 4, 2, 128, 16, 16), 0), (([300], [1], 4, 2, 128, 16, 16), 1),
                                       (([3000], [4], 8, 2, 128, 12, 4), 0), (([700], [9], 4, 2, 64, 32, 8), 3),
                                       (([500], [64], 4, 2, 128, 16, 16), 1), (([900, 20], [100, 70], 16, 8, 64, 12, 12), 0),
                                       (([9000], [64], 2, 1, 128, 16, 16), 2)])
def test_products_that_never_come(q3, case, tile, dtype):
    """A wait inside the kernel that runs out: reported within the limit, and the next
    calls are right."""
    import time
    import torch
    c = attend_case(np.random.default_rng(22), *case, dtype=dtype, tree=False)
    want = run_attention(q3, c)

    def run():
        status = ku.ints([0])
        out = run_attention(q3, c, status=status)
        return out, int(status)

    q3.debug_lose_tile(1 << 30, 2000000)  # no such tile
    out, code = run()
    assert code == 0 and torch.equal(out, want)
    for _ in range(2):
        q3.debug_lose_tile(tile, 2000)
        t0 = time.perf_counter()
        code = run()[1]
        # (a share of a split item may have fewer tiles than the item)
        assert code in ((q3.ERR_TIMEOUT,) if tile == 0 else (q3.ERR_TIMEOUT, 0)) and time.perf_counter() - t0 < 1.0
        out, code = run()
        assert code == 0 and torch.equal(out, want)
