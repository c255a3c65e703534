"""Measured cases of the 8-bit cache's operators: quantising keys and values as
they are written to a paged cache, reading them back, and the attention over it.

The cache is [layers][pages][k|v][kv heads][page positions][head dim] of FP8 E4M3
codes, with one power of two for each block of positions of a page, kv head and
k or v (an E8M0 byte b stands for 2^(b - 127)): an element is code x 2^(b - 127).
A block's power is the smallest that brings its largest finite magnitude to 448 or
below; while a block is being filled it only rises, and the codes that are already
there are rounded again to the new one.

With ``own`` false, ``run`` computes an operator from elementary torch operations
in 32 bits; with ``own`` true it makes the calls a user of the library makes.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "fp32"
CAUSAL, TREE = "causal", "tree"


# ------------------------------------------------------------------ cases
def _case(name, op, seqs, ctx_lo, ctx_hi, rows_lo, rows_hi, kv_heads=8, hd=128, page=16, block=16, dtype=F32, **more):
    return {"name": name, "op": op, "seqs": seqs, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "rows_lo": rows_lo,
            "rows_hi": rows_hi, "kv_heads": kv_heads, "hd": hd, "page": page, "block": block, "dtype": dtype, **more}


def _attend(name, seqs, ctx_lo, ctx_hi, rows_lo, rows_hi, heads=16, sees=CAUSAL, blind=False, **more):
    return _case(name, "attend", seqs, ctx_lo, ctx_hi, rows_lo, rows_hi, heads=heads, sees=sees, blind=blind, **more)


def listed():
    return [
        # one 1.7B stream's decode step: a position is appended inside a block; latency counts
        _case("write 1x131 single", "write", 1, 131, 131, 1, 1),
        # the serving batch's decode step: a position of every stream
        _case("write 128x256..2048 single", "write", 128, 256, 2048, 1, 1, dtype=BF16),
        # prompts of several streams in one call, some of them short, from any offset in a block
        _case("write 8x0..37 2..1982 rows", "write", 8, 0, 37, 2, 1982),
        # the accepted path of one stream's drafted tree, to be written where it belongs
        _case("read 1x131 path 4", "read", 1, 131, 131, 4, 4, path=True),
        # long contexts taken out whole, for a cache of another kind
        _case("read 4x0 30011..32768 rows", "read", 4, 0, 0, 30011, 32768, dtype=BF16, path=False),
        # one stream early in its episode, one token: latency counts
        _attend("attend 1x131 single", 1, 131, 131, 1, 1),
        # batched streams, one new frame each
        _attend("attend 16x32..512 single", 16, 32, 512, 1, 1, dtype=BF16),
        # the serving batch with its contexts
        _attend("attend 128x256..2048 single", 128, 256, 2048, 1, 1),
        # few streams far into long episodes, the largest drafted trees
        _attend("attend 4x30011..32768 tree 64", 4, 30011, 32768, 64, 64, sees=TREE),
        # the serving prompt from its first position
        _attend("attend 1x0 1982 rows", 1, 0, 0, 1982, 1982),
        # a chunk of a long prompt after the chunks before it
        _attend("attend 1x14336 2048 rows", 1, 14336, 14336, 2048, 2048, dtype=BF16),
        # the tiny shape's heads, odd lengths and ragged trees, pages and blocks of other sizes, rows that see nothing
        _attend("attend 5x0..777 tree hd64", 5, 0, 777, 3, 37, heads=4, kv_heads=2, hd=64, page=12, block=4, sees=TREE,
                blind=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["write", "write", "read", "attend", "attend", "attend", "attend"])
    hd, page = rng.choice([64, 128, 128]), rng.choice([8, 12, 16, 16, 16, 24, 32, 64])
    block = rng.choice([b for b in (1, 2, 4, 8, 12, 16, 16, 16, 32, 64) if page % b == 0])
    c = {"op": op, "kv_heads": rng.choice([1, 2, 4, 8]), "hd": hd, "page": page, "block": block,
         "dtype": rng.choice([F32, BF16])}
    if op != "attend":
        hi = _log(rng, 1, 2048)
        nhi = _log(rng, 1, 2048 if op == "write" else 8192)
        c.update(seqs=_log(rng, 1, max(1, min(128, 40000 // (hi + nhi)))), ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                 rows_lo=rng.randint(1, nhi), rows_hi=nhi)
        if op == "read":
            c["path"] = rng.random() < 0.5
        return c
    heads = c["kv_heads"] * rng.choice([1, 2, 2, 2, 4, 8])
    kind = rng.choice(["single", "single", "tree", "chunk"])
    hi = _log(rng, 1, 16384)
    nhi = 1 if kind == "single" else _log(rng, 2, 64 if kind == "tree" else 2048)
    most = min(128, 100000 // (hi + nhi), int(2e8 // (heads * nhi * (hi + nhi))))
    c.update(seqs=_log(rng, 1, max(1, most)), ctx_lo=rng.randint(0, hi), ctx_hi=hi, rows_lo=rng.randint(1, nhi),
             rows_hi=nhi, heads=heads, sees=TREE if kind == "tree" else CAUSAL,
             blind=kind == "tree" and rng.random() < 0.3)
    return c


# ----------------------------------------------------------------- inputs
def _spread(lo, hi, n):
    """n whole numbers from lo to hi in equal steps (a lone one is hi)."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _mixed(rng, lo, hi, n):
    v = _spread(lo, hi, n)
    return [v[i] for i in rng.permutation(n)]


def _table(rng, lens, page):
    """A page table over a pool of a few more pages than any order of the lengths needs, in random order."""
    need = [max(1, -(-n // page)) for n in lens]
    pages = sum(lens) // page + len(lens) + 3
    perm, at = rng.permutation(pages), 0
    table = np.zeros((len(lens), max(need)), np.int32)
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    return pages, table


def _power(top):
    """The E8M0 byte of a block from its largest magnitude (fp32): 448 x 2^(byte - 127) is the least that holds it."""
    bits = top.contiguous().view(torch.int32)
    return (((bits + 0x1fffff) >> 23) - 8).clamp_(min=0)


def _two_to(byte):
    """2^(byte - 127) as fp32 (bytes below 255)."""
    return torch.where(byte > 0, byte << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _cache(case, pages, gen):
    """A filled cache of two layers: normal keys and values whose size differs from head to head and page to page."""
    shape = (2, pages, 2, case["kv_heads"], case["page"] // case["block"], case["block"], case["hd"])
    pool = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(shape[:5], dtype=torch.uint8, device="cuda")
    for layer in range(2):
        x = torch.randn(shape[1:], device="cuda", generator=gen)
        x *= torch.randn(shape[1:5] + (1, 1), device="cuda", generator=gen).mul_(0.5).exp_()
        byte = _power(x.abs().amax((-2, -1)))
        pool[layer] = (x * _two_to(254 - byte)[..., None, None]).to(torch.float8_e4m3fn)
        scales[layer] = byte.to(torch.uint8)
    return (pool.reshape(2, pages, 2, case["kv_heads"], case["page"], case["hd"]),
            scales.view(torch.float8_e8m0fnu))


def _parents(rng, n):
    """A drafted tree in the order it was drafted: node i hangs from an earlier node or from the context."""
    return [-1 if i == 0 else int(rng.integers(-1 if rng.random() < 0.3 else max(-1, i - 4), i)) for i in range(n)]


def _masks(case, rng, rows):
    masks = []
    for n in rows:
        own_bits = []
        for i, p in enumerate(_parents(rng, n)):
            own_bits.append((1 << i) | (own_bits[p] if p >= 0 else 0))
        masks += [0 if case["blind"] and rng.random() < 0.2 else m for m in own_bits]
    return torch.from_numpy(np.array(masks, np.uint64).view(np.int64)).cuda()


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(int(seed) + 1)
    dev = {"device": "cuda"}
    lens = _mixed(rng, case["ctx_lo"], case["ctx_hi"], case["seqs"])
    rows = _mixed(rng, case["rows_lo"], case["rows_hi"], case["seqs"])
    total, most = sum(rows), max(rows)
    # a path picks among a few more positions than it has
    ahead = [n + n // 2 + 3 if case.get("path") else n for n in rows]
    pages, table = _table(rng, [a + b for a, b in zip(lens, ahead)], case["page"])
    pool, scales = _cache(case, pages, gen)
    s = {"case": case, "pool": pool, "scales": scales, "table": torch.from_numpy(table).cuda(),
         "lengths": torch.tensor(lens, dtype=torch.int32, **dev),
         "start": torch.tensor(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32), **dev), "most": most}
    dtype = torch.bfloat16 if case["dtype"] == BF16 else torch.float32
    heads, hd = case["kv_heads"], case["hd"]
    if case["op"] == "write":
        # rows of a projection's output, [q | k | v]: views with its pitch
        qkv = torch.randn((total, 4 * heads, hd), generator=gen, **dev).to(dtype)
        s.update(k=qkv[:, 2 * heads:3 * heads], v=qkv[:, 3 * heads:])
    elif case["op"] == "read":
        path = [np.sort(rng.permutation(a)[:n]) for a, n in zip(ahead, rows)]
        s["path"] = torch.from_numpy(np.concatenate(path).astype(np.int32)).cuda() if case["path"] else None
        s["out"] = tuple(torch.empty((total, heads, hd), dtype=dtype, **dev) for _ in range(2))
    else:
        s["q"] = torch.randn((total, case["heads"], hd), generator=gen, **dev).to(dtype)
        s["out"] = torch.empty_like(s["q"])
        s["masks"] = _masks(case, rng, rows) if case["sees"] == TREE else None
    return s


# ------------------------------------------------------------- plain forms
def _rows(s, offsets=None):
    """(sequence, page, slot) of every row."""
    start, page = s["start"].long(), s["case"]["page"]
    row = torch.arange(int(s["k" if s["case"]["op"] == "write" else "q"].shape[0]) if offsets is None else offsets.numel(),
                       device=start.device)
    seq = torch.searchsorted(start[1:], row, right=True)
    pos = s["lengths"].long()[seq] + (row - start[seq] if offsets is None else offsets.long())
    return seq, pos, s["table"].long()[seq, pos // page], pos % page


def _plain_write(s):
    case, pool, scales = s["case"], s["pool"][1], s["scales"].view(torch.uint8)[1]
    block, page, hd = case["block"], case["page"], case["hd"]
    seq, pos, at, slot = _rows(s)
    x = torch.stack([s["k"], s["v"]], 1).float()  # [rows, 2, kv heads, hd]
    size = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    # blocks of a sequence, numbered on from the first that it writes to
    blocks = page * s["table"].shape[1] // block
    which, of = torch.unique(seq * blocks + pos // block, return_inverse=True)
    top = torch.zeros((which.numel(),) + size.shape[1:], device=x.device)
    top.scatter_reduce_(0, of[:, None, None].expand_as(size), size, "amax")
    byte = _power(top)
    wseq, wpos = which // blocks, which % blocks * block  # a block's sequence and first position
    wat, wsub = s["table"].long()[wseq, wpos // page], wpos % page // block
    held = (s["lengths"].long()[wseq] - wpos).clamp(min=0)  # rows of it that were there before
    before = scales[wat, :, :, wsub].int()
    byte = torch.where((held > 0)[:, None, None], torch.maximum(byte, before), byte)
    lanes = torch.arange(block, device=x.device)
    codes = pool.view(-1, 2, case["kv_heads"], page // block, block, hd)
    old = codes[wat, :, :, wsub].float()
    again = (old * _two_to((before - byte + 127).clamp(min=0))[..., None, None]).to(torch.float8_e4m3fn)
    keep = ((lanes[None, :] < held[:, None])[:, None, None] & (byte > before)[..., None])[..., None]
    codes[wat, :, :, wsub] = torch.where(keep, again.view(torch.uint8), codes[wat, :, :, wsub].view(torch.uint8)).view(
        torch.float8_e4m3fn)
    scales[wat, :, :, wsub] = byte.to(torch.uint8)
    pool[at, :, :, slot] = (x * _two_to(254 - byte)[of][..., None]).to(torch.float8_e4m3fn)
    return s["pool"], s["scales"]


def _values(s, at, slot):
    """Keys and values of the positions as fp32, [.., 2, kv heads, hd]."""
    byte = s["scales"].view(torch.uint8)[1][at, :, :, slot // s["case"]["block"]].int()
    return s["pool"][1][at, :, :, slot].float() * _two_to(byte)[..., None]


def _plain_read(s):
    offsets = s["path"]
    if offsets is None:
        start = s["start"].long()
        row = torch.arange(s["out"][0].shape[0], device=start.device)
        offsets = row - start[torch.searchsorted(start[1:], row, right=True)]
    _, _, at, slot = _rows(s, offsets)
    x = _values(s, at, slot)
    s["out"][0].copy_(x[:, 0])
    s["out"][1].copy_(x[:, 1])
    return s["out"]


def _plain_attend(s):
    case, start, q = s["case"], s["start"].long(), s["q"].float()
    total, heads, hd = q.shape
    seqs, n, kvh, page = s["lengths"].numel(), s["most"], case["kv_heads"], case["page"]
    byte = s["scales"].view(torch.uint8)[1][s["table"].long()].int()  # [seqs, pages, 2, kv heads, blocks]
    kv = s["pool"][1][s["table"].long()].float()
    kv = kv * _two_to(byte).repeat_interleave(case["block"], -1)[..., None]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, seqs, kvh, -1, hd)
    span = kv.shape[3]
    rows = start[1:] - start[:-1]
    row = start[:-1, None] + torch.arange(n, device=q.device)
    live = row < start[1:, None]
    row = row.clamp(max=total - 1)
    off = torch.arange(span, device=q.device)[None, :] - s["lengths"].long()[:, None]  # the row a position holds
    if s["masks"] is not None:
        bit = (s["masks"][row][:, :, None] >> off[:, None].clamp(0, 63)) & 1
        sees = (off < 0)[:, None] | ((off < n)[:, None] & (bit != 0))
    else:
        sees = off[:, None] <= torch.arange(n, device=q.device)[None, :, None]
    sees = sees & live[:, :, None]
    kv = torch.where((off < rows[:, None])[None, :, None, :, None], kv, torch.zeros((), device=q.device))
    qs = q[row].reshape(seqs, n, kvh, heads // kvh, hd).permute(0, 2, 3, 1, 4).reshape(seqs, kvh, -1, hd)
    sc = (qs @ kv[0].transpose(-1, -2)).mul_(1.0 / math.sqrt(hd)).view(seqs, kvh, heads // kvh, n, span)
    sees = sees[:, None, None]
    sc = torch.where(sees, sc, torch.full((), -math.inf, device=q.device))
    top = sc.amax(-1, keepdim=True)
    p = (sc - torch.where(torch.isneginf(top), 0.0, top)).exp_()
    z = p.sum(-1)[..., None]
    o = (p.view(seqs, kvh, -1, span) @ kv[1]).view(seqs, kvh, heads // kvh, n, hd)
    o = torch.where(z > 0, o / z, 0.0).permute(0, 3, 1, 2, 4).reshape(seqs, n, heads, hd)
    s["out"][row[live]] = o[live].to(s["out"].dtype)
    return s["out"]


def run(s):
    op = s["case"]["op"]
    if own:
        from autoregressive_tts_decode_gb300 import q3tts
        cache = s["pool"], s["scales"], 1, s["table"], s["lengths"], s["start"]
        if op == "write":
            q3tts.kv8_write(*cache, s["k"], s["v"], max_rows=s["most"])
            return s["pool"], s["scales"]
        if op == "read":
            return q3tts.kv8_read(*cache, path=s["path"], max_rows=s["most"], out=s["out"])
        return q3tts.kv8_attention(*cache, s["q"], masks=s["masks"], max_rows=s["most"], out=s["out"])
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[op](s)


# ------------------------------------------------------------ what it costs
def work(case):
    lens, rows = (_spread(case[k + "_lo"], case[k + "_hi"], case["seqs"]) for k in ("ctx", "rows"))
    width, size = 2 * case["kv_heads"] * case["hd"], 2 if case["dtype"] == BF16 else 4
    blocks = lambda n: 2 * case["kv_heads"] * -(-n // case["block"])  # noqa: E731
    if case["op"] != "attend":
        # rows in one form, codes and powers in the other, page ids and lengths
        total = sum(rows)
        moved = total * width * (size + 1) + sum(blocks(n) for n in rows)
        return {"bytes": moved + 4 * sum(-(-n // case["page"]) for n in rows) + 8 * case["seqs"] + 4 * total * bool(case.get("path")),
                "flops": 0}
    q = case["heads"] * case["hd"]
    # which length meets which rows is up to the seed: the average
    pairs = sum(rows) * sum(lens) / case["seqs"] + sum(n * (n + 1) / 2 for n in rows)
    return {"bytes": sum(lens + rows) * width + sum(map(blocks, lens)) + sum(rows) * (2 * q * size + (8 if case["sees"] == TREE else 0)) +
            4 * sum(-(-n // case["page"]) for n in lens), "flops": 4.0 * q * pairs}


# ------------------------------------------------- 64 bits, written apart
def _e4m3(y):
    """y (64 bits, at most 448 in size) to the nearest E4M3 value, ties to the even one."""
    _, e = torch.frexp(y)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(y / step) * step


def _exact_write(case, s):
    pool, scales = s["pool"].double(), torch.exp2(s["scales"].view(torch.uint8).double() - 127)
    start, table, lens = s["start"].tolist(), s["table"].tolist(), s["lengths"].tolist()
    page, block = case["page"], case["block"]
    for i, length in enumerate(lens):
        at, end = length, length + start[i + 1] - start[i]
        while at < end:
            stop = min(end, (at // block + 1) * block)
            first = at // block * block
            a, b = start[i] + at - length, start[i] + stop - length
            p, sub = table[i][at // page], at % page // block
            for j, src in enumerate((s["k"], s["v"])):
                x = src[a:b].double().transpose(0, 1)  # [kv heads, rows, hd]
                top = x.abs().amax((1, 2))
                two = torch.exp2(torch.ceil(torch.log2(top / 448)))  # the powers here are far from either end
                old = scales[1, p, j, :, sub]
                if at > first:  # rows from before: the power does not fall
                    two = torch.maximum(two, old)
                    slots = slice(first % page, at % page)
                    pool[1, p, j, :, slots] = _e4m3(pool[1, p, j, :, slots] * (old / two)[:, None, None])
                pool[1, p, j, :, at % page:at % page + stop - at] = _e4m3(x / two[:, None, None])
                scales[1, p, j, :, sub] = two
            at = stop
    return pool, scales


def _exact_values(case, s, i, pos):
    """Keys and values of sequence i's positions, [2, positions, kv heads, hd]."""
    page, slot = s["table"][i].long()[pos // case["page"]], pos % case["page"]
    two = torch.exp2(s["scales"].view(torch.uint8)[1].double() - 127)
    return torch.stack([s["pool"][1, page, j, :, slot].double() * two[page, j, :, slot // case["block"]][..., None]
                        for j in (0, 1)])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(case, s)
    start, lens = s["start"].tolist(), s["lengths"].tolist()
    if case["op"] == "read":
        got = []
        for i, length in enumerate(lens):
            n = start[i + 1] - start[i]
            off = torch.arange(n, device="cuda") if s["path"] is None else s["path"][start[i]:start[i + 1]].long()
            got.append(_exact_values(case, s, i, length + off))
        kv = torch.cat(got, 1)
        return kv[0], kv[1]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    rep = case["heads"] // case["kv_heads"]
    for i, length in enumerate(lens):
        a, b = start[i], start[i + 1]
        n = b - a
        k, v = _exact_values(case, s, i, torch.arange(length + n, device="cuda"))
        ok = torch.ones((n, length + n), dtype=torch.bool, device="cuda")
        if s["masks"] is None:
            ok[:, length:] = torch.ones((n, n), device="cuda").tril() > 0
        else:
            for j in range(n):
                ok[:, length + j] = ((s["masks"][a:b] >> j) & 1) != 0
        for h in range(case["heads"]):
            w = (s["q"][a:b, h].double() @ k[:, h // rep].T) / case["hd"] ** 0.5
            w = torch.softmax(w.masked_fill(~ok, -math.inf), -1)
            out[a:b, h] = torch.where(ok.any(-1, keepdim=True), w, 0.0) @ v[:, h // rep]
    return out
