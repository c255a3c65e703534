"""Measured cases of the branching-decode operators: attention of drafted trees
over a paged cache, copies and compaction of cache pages, and beam selection
with its reordering of states.

The cache is the engine's: [layers][pages][k|v][kv heads][page positions][head
dim], bf16 or fp32, a page holding one position range of a sequence in every
layer.  With ``own`` false, ``run`` computes an operator from elementary torch
operations in 32 bits (64 where scores are compared); with ``own`` true it makes
the calls a user of the library makes.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "fp32"


# ------------------------------------------------------------------ cases
def _tree(name, seqs, ctx_lo, ctx_hi, nodes_lo, nodes_hi, heads=16, kv_heads=8, hd=128, page=16, kv=BF16):
    return {"name": name, "op": "tree", "seqs": seqs, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "nodes_lo": nodes_lo,
            "nodes_hi": nodes_hi, "heads": heads, "kv_heads": kv_heads, "hd": hd, "page": page, "kv": kv}


def _copy(name, pairs, layers, pages, kv_heads=8, hd=128, page=16, kv=BF16):
    return {"name": name, "op": "copy", "pairs": pairs, "layers": layers, "pages": pages, "kv_heads": kv_heads,
            "hd": hd, "page": page, "kv": kv}


def _compact(name, seqs, layers, ctx_lo, ctx_hi, nodes, accept_lo, accept_hi, kv_heads=8, hd=128, page=16, kv=BF16):
    return {"name": name, "op": "compact", "seqs": seqs, "layers": layers, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "nodes": nodes, "accept_lo": accept_lo, "accept_hi": accept_hi, "kv_heads": kv_heads, "hd": hd,
            "page": page, "kv": kv}


def _beam(name, groups, beams, k, vocab, hidden, history, finished):
    return {"name": name, "op": "beam", "groups": groups, "beams": beams, "k": k, "vocab": vocab, "hidden": hidden,
            "history": history, "finished": finished}


def listed():
    return [
        # one 1.7B stream early in its episode checks eight drafted frames: latency counts
        _tree("tree 1x131 8 nodes", 1, 131, 131, 8, 8),
        # the form for single tokens: batched streams, one new frame each
        _tree("tree 16x32..512 single", 16, 32, 512, 1, 1),
        # the serving batch with its contexts, a tree for each stream
        _tree("tree 128x256..2048 16 nodes", 128, 256, 2048, 16, 16),
        # few streams far into long episodes, the largest tree
        _tree("tree 4x30011..32768 64 nodes", 4, 30011, 32768, 64, 64),
        # the tiny shape's heads and fp32 cache, odd lengths and ragged trees
        _tree("tree 5x1..777 fp32 hd64", 5, 1, 777, 3, 37, heads=4, kv_heads=2, hd=64, kv=F32),
        # a prompt forked for three more takes: the last, partly filled page is copied
        _copy("copy 3 pages", 3, 28, 96),
        # every page of several long streams moved at once
        _copy("copy 300 pages", 300, 28, 640),
        # the accepted path of one stream's tree becomes its context
        _compact("compact 1x131 4 of 8", 1, 28, 131, 131, 8, 4, 4),
        # the same for a batch of streams, ragged paths among them empty ones
        _compact("compact 64x32..256 0..12 of 16", 64, 28, 32, 256, 16, 0, 12),
        # one utterance searched with four beams, semantic codes up to the engine's largest vocabulary
        _beam("beam 1x4 of 4096", 1, 4, 4, 4096, 2048, True, False),
        # thirty-two utterances with four beams each: the serving batch
        _beam("beam 32x4 of 2048", 32, 4, 4, 2048, 2048, True, True),
        # wide beams over a text-sized vocabulary
        _beam("beam 8x16 of 131072", 8, 16, 16, 131072, 2048, False, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "copy", "compact", "beam", "beam"])
    kv = BF16 if rng.random() < 0.75 else F32
    hd, page = rng.choice([64, 128]), rng.choice([8, 12, 16, 16, 16, 32, 64])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "tree":
        hi = _log(rng, 1, 16384)
        lo = rng.randint(0, hi)
        seqs = _log(rng, 1, max(1, min(128, 100000 // hi)))
        nhi = _log(rng, 1, 64)
        return {"op": op, "seqs": seqs, "ctx_lo": lo, "ctx_hi": hi, "nodes_lo": rng.randint(1, nhi), "nodes_hi": nhi,
                "heads": kv_heads * rng.choice([1, 2, 2, 4]), "kv_heads": kv_heads, "hd": hd, "page": page, "kv": kv}
    if op == "copy":
        layers = _log(rng, 1, 32)
        pairs = _log(rng, 1, 250)
        return {"op": op, "pairs": pairs, "layers": layers, "pages": 2 * pairs + rng.randint(0, 100),
                "kv_heads": kv_heads, "hd": hd, "page": rng.choice([8, 12, 16]), "kv": kv}
    if op == "compact":
        hi = _log(rng, 1, 2048)
        nodes = _log(rng, 2, 64)
        ahi = rng.randint(1, nodes - 1)
        return {"op": op, "seqs": _log(rng, 1, max(1, min(128, 16000 // (hi + nodes)))), "layers": _log(rng, 1, 28),
                "ctx_lo": rng.randint(0, hi), "ctx_hi": hi, "nodes": nodes, "accept_lo": rng.randint(0, ahi),
                "accept_hi": ahi, "kv_heads": kv_heads, "hd": hd, "page": page, "kv": kv}
    beams = _log(rng, 1, 32)
    vocab = _log(rng, 64, 131072)
    return {"op": op, "groups": _log(rng, 1, max(1, min(64, 16000000 // (beams * vocab)))), "beams": beams,
            "k": rng.randint(1, beams), "vocab": vocab, "hidden": 8 * _log(rng, 8, 512), "history": rng.random() < 0.5,
            "finished": rng.random() < 0.5}


# ----------------------------------------------------------------- inputs
def _spread(lo, hi, n):
    """n whole numbers from lo to hi in equal steps (a lone one is hi)."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _dtype(kv):
    return torch.bfloat16 if kv == BF16 else torch.float32


def _pool(case, layers, pages, gen):
    shape = (layers, pages, 2, case["kv_heads"], case["page"], case["hd"])
    return torch.randn(shape, device="cuda", generator=gen, dtype=_dtype(case["kv"]))


def _table(rng, lens, page):
    """A page table over a pool of a few more pages than the lengths need, in random order."""
    need = [max(1, -(-n // page)) for n in lens]
    pages = sum(need) + 3
    perm, at = rng.permutation(pages), 0
    table = np.zeros((len(lens), max(need)), np.int32)
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    return pages, table


def _parents(rng, n):
    """A drafted tree in the order it was drafted: node i hangs from an earlier node or from the context."""
    return [-1 if i == 0 else int(rng.integers(-1 if rng.random() < 0.3 else max(-1, i - 4), i)) for i in range(n)]


def _ragged(case, rng):
    lens = _spread(case["ctx_lo"], case["ctx_hi"], case["seqs"])
    return [lens[i] for i in rng.permutation(len(lens))]


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(int(seed) + 1)
    dev = {"device": "cuda"}
    if case["op"] == "tree":
        lens = _ragged(case, rng)
        nodes = _spread(case["nodes_lo"], case["nodes_hi"], case["seqs"])
        nodes = [nodes[i] for i in rng.permutation(len(nodes))]
        pages, table = _table(rng, [a + b for a, b in zip(lens, nodes)], case["page"])
        masks = []
        for n in nodes:
            own_bits = []
            for i, p in enumerate(_parents(rng, n)):
                own_bits.append((1 << i) | (own_bits[p] if p >= 0 else 0))
            masks += own_bits
        total = len(masks)
        return {
            "case": case,
            "pool": _pool(case, 2, pages, gen),
            "table": torch.from_numpy(table).cuda(),
            "lengths": torch.tensor(lens, dtype=torch.int32, **dev),
            "start": torch.tensor(np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32), **dev),
            "masks": torch.from_numpy(np.array(masks, np.uint64).view(np.int64)).cuda(),
            "q": torch.randn((total, case["heads"], case["hd"]), generator=gen, **dev),
            "out": torch.empty((total, case["heads"], case["hd"]), **dev),
            "max_nodes": max(nodes),
        }
    if case["op"] == "copy":
        perm = rng.permutation(case["pages"])[:2 * case["pairs"]].astype(np.int32)
        return {"case": case, "pool": _pool(case, case["layers"], case["pages"], gen),
                "src": torch.from_numpy(perm[:case["pairs"]].copy()),
                "dst": torch.from_numpy(perm[case["pairs"]:].copy())}
    if case["op"] == "compact":
        lens = _ragged(case, rng)
        pages, table = _table(rng, [n + case["nodes"] for n in lens], case["page"])
        counts = _spread(case["accept_lo"], case["accept_hi"], case["seqs"])
        path = np.zeros((case["seqs"], case["nodes"]), np.int32)
        for s, n in enumerate(counts):  # an ascending path that leaves out node 0: every accepted row moves
            path[s, :n] = np.sort(rng.permutation(case["nodes"] - 1)[:n] + 1)
        return {"case": case, "pool": _pool(case, case["layers"], pages, gen), "table": torch.from_numpy(table).cuda(),
                "lengths": torch.tensor(lens, dtype=torch.int32, **dev), "path": torch.from_numpy(path).cuda(),
                "path_len": torch.tensor(counts, dtype=torch.int32, **dev)}
    g, b, v, h = case["groups"], case["beams"], case["vocab"], case["hidden"]
    hist = (torch.rand((g, b, v), generator=gen, **dev) < 0.05).to(torch.uint8) if case["history"] else None
    done = (torch.rand((g, b), generator=gen, **dev) < 0.15).to(torch.uint8) if case["finished"] else None
    rows = [torch.randn((g, b, h), generator=gen, **dev)] + ([hist] if case["history"] else [])
    return {"case": case, "logits": torch.randn((g, b, v), generator=gen, **dev) * 3.0,
            "scores": -20.0 * torch.rand((g, b), generator=gen, **dev), "history": hist, "finished": done,
            "rows": rows, "next": [torch.empty((g, case["k"]) + tuple(r.shape[2:]), dtype=r.dtype, **dev) for r in rows],
            "eos": v - 1, "special": v - max(2, v // 16), "penalty": 1.05}


# ------------------------------------------------------------- plain forms
def _plain_tree(s):
    pool, start, q = s["pool"][1], s["start"].long(), s["q"].float()
    total, heads, hd = q.shape
    seqs, n = s["lengths"].numel(), s["max_nodes"]
    kvh, page = pool.shape[2], pool.shape[3]
    pages = pool[s["table"].long()].float()  # [seqs, pages, 2, kv heads, page, hd]
    kv = pages.permute(2, 0, 3, 1, 4, 5).reshape(2, seqs, kvh, -1, hd)
    span = kv.shape[3]
    row = start[:-1, None] + torch.arange(n, device=q.device)
    live = row < start[1:, None]
    row = row.clamp(max=total - 1)
    lens = s["lengths"].long()[:, None, None]
    off = torch.arange(span, device=q.device)[None, None, :] - lens  # the node a position holds
    bit = (s["masks"][row][:, :, None] >> off.clamp(0, 63)) & 1
    sees = (off < 0) | ((off < n) & (bit != 0))
    sees = sees & live[:, :, None]
    held = (off < (start[1:] - start[:-1])[:, None, None]).squeeze(1)
    kv = torch.where(held[None, :, None, :, None], kv, torch.zeros((), device=q.device))
    qs = q[row].reshape(seqs, n, kvh, heads // kvh, hd).permute(0, 2, 1, 3, 4).reshape(seqs, kvh, -1, hd)
    sc = qs @ kv[0].transpose(-1, -2) * (1.0 / math.sqrt(hd))
    sees = sees[:, None, :, None, :].expand(seqs, kvh, n, heads // kvh, span).reshape(sc.shape)
    sc = torch.where(sees, sc, torch.full((), -math.inf, device=q.device))
    top = sc.amax(-1, keepdim=True)
    p = torch.where(sees, (sc - torch.where(sees.any(-1, keepdim=True), top, 0.0)).exp(), 0.0)
    z = p.sum(-1, keepdim=True)
    o = torch.where(z > 0, (p @ kv[1]) / z, 0.0)
    o = o.reshape(seqs, kvh, n, heads // kvh, hd).permute(0, 2, 1, 3, 4).reshape(seqs, n, heads, hd)
    s["out"][row[live]] = o[live]
    return s["out"]


def _plain_copy(s):
    src, dst = s["src"].cuda().long(), s["dst"].cuda().long()
    s["pool"][:, dst] = s["pool"][:, src]
    return s["pool"]


def _plain_compact(s):
    pool, page = s["pool"], s["pool"].shape[4]
    i = torch.arange(s["path"].shape[1], device=pool.device)
    seq, i = torch.nonzero(i[None, :] < s["path_len"][:, None], as_tuple=True)
    to = s["lengths"].long()[seq] + i
    of = s["lengths"].long()[seq] + s["path"].long()[seq, i]
    table = s["table"].long()
    pool[:, table[seq, to // page], :, :, to % page] = pool[:, table[seq, of // page], :, :, of % page].clone()
    return pool


def _plain_beam(s):
    c = s["case"]
    g, b, v, k = c["groups"], c["beams"], c["vocab"], c["k"]
    x = s["logits"]
    if s["history"] is not None:
        x = torch.where(s["history"] != 0, torch.where(x > 0, x / s["penalty"], x * s["penalty"]), x)
    tok = torch.arange(v, device=x.device)
    x = torch.where((tok >= s["special"]) & (tok != s["eos"]), -math.inf, x)
    x, tok = torch.sort(x, dim=-1, descending=True, stable=True)
    y = x.double()
    z = (y - y[..., :1]).exp().sum(-1, keepdim=True).log()
    score = s["scores"].double()[..., None] + ((y - y[..., :1]) - z)
    if s["finished"] is not None:  # a finished beam stays as it is: one candidate, its end token
        done = s["finished"][..., None] != 0
        first = torch.arange(v, device=x.device) == 0
        score = torch.where(done, torch.where(first, s["scores"].double()[..., None], -math.inf), score)
        tok = torch.where(done, s["eos"], tok)
    score, at = torch.sort(score.reshape(g, -1), dim=-1, descending=True, stable=True)
    score, at = score[:, :k], at[:, :k]
    none = torch.isneginf(score)  # no candidate left for the slot
    tokens = torch.where(none, -1, tok.reshape(g, -1).gather(1, at)).int()
    parents = torch.where(none, 0, at // v).int()
    nxt = [r[torch.arange(g, device=x.device)[:, None], parents.long()] for r in s["rows"]]
    return {"tokens": tokens, "parents": parents, "scores": score.float(), "rows": nxt}


def run(s):
    op = s["case"]["op"]
    if own:
        from autoregressive_tts_decode_gb300 import q3tts
        if op == "tree":
            return q3tts.tree_attention(s["pool"], 1, s["table"], s["lengths"], s["start"], s["masks"], s["q"],
                                        max_nodes=s["max_nodes"], out=s["out"])
        if op == "copy":
            return q3tts.copy_pages(s["pool"], s["src"], s["dst"])
        if op == "compact":
            return q3tts.compact_rows(s["pool"], s["table"], s["lengths"], s["path"], s["path_len"])
        tokens, parents, scores = q3tts.beam_select(
            s["logits"], s["scores"], k=s["case"]["k"], history=s["history"], finished=s["finished"],
            eos_token=s["eos"], special_from=s["special"], repetition_penalty=s["penalty"])
        q3tts.reorder_rows(s["rows"], s["next"], parents)
        return {"tokens": tokens, "parents": parents, "scores": scores, "rows": s["next"]}
    return {"tree": _plain_tree, "copy": _plain_copy, "compact": _plain_compact, "beam": _plain_beam}[op](s)


# ------------------------------------------------------------ what it costs
def work(case):
    if case["op"] == "beam":
        g, b, v, k = case["groups"], case["beams"], case["vocab"], case["k"]
        row = case["hidden"] * 4 + (v if case["history"] else 0)
        read = g * b * (v * (5 if case["history"] else 4) + 4)
        return {"bytes": read + g * k * (12 + 2 * row), "flops": 4.0 * g * b * v}
    row = 2 * case["kv_heads"] * case["hd"] * (2 if case["kv"] == BF16 else 4)  # k and v of one position
    if case["op"] == "copy":
        return {"bytes": 2 * case["pairs"] * case["layers"] * case["page"] * row, "flops": 0}
    if case["op"] == "compact":
        moved = sum(_spread(case["accept_lo"], case["accept_hi"], case["seqs"]))
        return {"bytes": 2 * moved * case["layers"] * row + case["seqs"] * 8 + 4 * moved, "flops": 0}
    lens, nodes = (_spread(case[k + "_lo"], case[k + "_hi"], case["seqs"]) for k in ("ctx", "nodes"))
    q = case["heads"] * case["hd"]
    # which length meets which tree is up to the seed: the average
    pairs = sum(nodes) * sum(lens) / case["seqs"] + sum(n * (n + 1) / 2 for n in nodes)
    return {"bytes": sum(lens + nodes) * row + sum(nodes) * (8 * q + 8) + sum(-(-n // case["page"]) for n in lens) * 4,
            "flops": 4.0 * q * pairs}


# ------------------------------------------------- 64 bits, written apart
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        start, lens = s["start"].tolist(), s["lengths"].tolist()
        rep = case["heads"] // case["kv_heads"]
        for i, length in enumerate(lens):
            a, b = start[i], start[i + 1]
            pos = torch.arange(length + b - a, device="cuda")
            page, slot = s["table"][i].long()[pos // case["page"]], pos % case["page"]
            k, v = (s["pool"][1, page, j, :, slot].double() for j in (0, 1))  # [positions, kv heads, hd]
            ok = torch.ones((b - a, length + b - a), dtype=torch.bool, device="cuda")
            for j in range(b - a):
                ok[:, length + j] = ((s["masks"][a:b] >> j) & 1) != 0
            for h in range(case["heads"]):
                w = (s["q"][a:b, h].double() @ k[:, h // rep].T) / case["hd"] ** 0.5
                out[a:b, h] = torch.softmax(w.masked_fill(~ok, -math.inf), -1) @ v[:, h // rep]
        return out
    if case["op"] == "copy":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            s["pool"][:, b].copy_(s["pool"][:, a])
        return s["pool"]
    if case["op"] == "compact":
        table, lens = s["table"].tolist(), s["lengths"].tolist()
        for i, n in enumerate(s["path_len"].tolist()):
            for to, of in enumerate(s["path"][i, :n].tolist()):  # ascending: a row is read before it is written over
                (p, a), (r, b) = divmod(lens[i] + of, case["page"]), divmod(lens[i] + to, case["page"])
                s["pool"][:, table[i][r], :, :, b] = s["pool"][:, table[i][p], :, :, a]
        return s["pool"]
    g, b, v, k = case["groups"], case["beams"], case["vocab"], case["k"]
    x = s["logits"].clone()
    if case["history"]:
        seen = s["history"] != 0
        x[seen & (x > 0)] /= s["penalty"]
        x[seen & (s["logits"] <= 0)] *= s["penalty"]
    end = x[:, :, s["eos"]].clone()
    x[:, :, s["special"]:] = -math.inf
    x[:, :, s["eos"]] = end
    lp = torch.log_softmax(x.double(), -1) + s["scores"].double()[:, :, None]
    if case["finished"]:
        for gi, bi in torch.nonzero(s["finished"]).tolist():
            lp[gi, bi] = -math.inf
            lp[gi, bi, s["eos"]] = s["scores"][gi, bi].double()
    best, at = torch.topk(lp.reshape(g, -1), k, dim=-1)
    parents = at // v
    rows = [torch.stack([r[i].index_select(0, parents[i]) for i in range(g)]) for r in s["rows"]]
    return {"tokens": at % v, "parents": parents, "scores": best, "rows": rows}
