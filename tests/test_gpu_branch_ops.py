"""The branching-decode operators on the GPU against their definitions in 64
bits: tree attention, page copies, compaction, beam selection, reordering, and
the five of them together as a search uses them."""
import math

import numpy as np
import pytest

from tests import branch_util as bu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from autoregressive_tts_decode_gb300 import build, q3tts
    build.build()
    return q3tts


def tree_case(rng, lens, nodes, heads, kv_heads, hd, page, dtype, layers=2, parents=None):
    import torch
    pool, table = bu.paged_cache(rng, [a + b for a, b in zip(lens, nodes)], page, layers, kv_heads, hd, dtype)
    masks = []
    for i, n in enumerate(nodes):
        masks += bu.tree_masks(parents[i] if parents else bu.tree_parents(rng, n))
    start = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    gen = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 31)))
    q = torch.randn((len(masks), heads, hd), generator=gen, device="cuda")
    return dict(pool=pool, table=table, lens=lens, nodes=nodes, masks=masks, q=q,
                lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"), start=torch.from_numpy(start).cuda())


def run_tree(q3, c, layer=1, **kw):
    return q3.tree_attention(c["pool"], layer, c["table"], c["lengths"], c["start"], bu.masks_tensor(c["masks"]),
                             c["q"], max_nodes=max(1, max(c["nodes"])), **kw)


def check_tree(c, out, layer=1):
    want, tol = bu.tree_reference(c["pool"], layer, c["table"], c["lens"], c["nodes"], c["masks"], c["q"])
    off = (out.double() - want).abs() / tol
    assert bool((off <= 1).all()), f"{float(off.max()):.3g} of the bound"


TREES = [
    # lens, nodes, heads, kv heads, head dim, page
    ([0], [1], 2, 1, 64, 16), ([1], [1], 4, 2, 128, 16), ([0], [64], 2, 1, 128, 16),
    ([131], [8], 16, 8, 128, 16), ([127, 128, 129], [1, 1, 1], 4, 2, 128, 16),
    ([15, 16, 17, 0], [1, 16, 17, 3], 4, 2, 64, 16), ([100, 0, 50], [0, 5, 0], 4, 2, 128, 16),
    ([777, 3, 260], [64, 1, 33], 8, 2, 128, 16), ([500], [9], 3, 3, 64, 12), ([200, 31], [7, 2], 8, 1, 128, 8),
    ([300], [20], 12, 3, 128, 32), ([129], [5], 4, 2, 64, 64), ([511], [40], 4, 4, 64, 128),
    ([600], [13], 4, 2, 128, 256), ([70], [64], 16, 1, 64, 16), ([45], [6], 2, 1, 128, 1),
    ([2048], [16], 16, 8, 128, 16), ([5000, 1], [3, 3], 2, 1, 64, 16), ([333], [17], 10, 2, 128, 24),
    # more than 64 rows to a kv head: few heads and sequences, then many
    ([9000], [64], 4, 2, 128, 16), ([960, 3, 0], [64, 33, 40], 16, 2, 128, 16), ([383], [22], 3, 1, 64, 256),
    ([9000, 0, 700, 5000] * 4, [64, 40, 33, 1] * 4, 4, 2, 128, 16), ([383] * 19, [22] * 19, 24, 8, 64, 256),
    ([127, 64, 0, 200] * 20, [64, 64, 64, 10] * 20, 4, 2, 128, 8), ([700, 3, 0, 260] * 3, [64, 33, 40, 0] * 3, 16, 2, 128, 16),
    ([500, 129] * 12, [64, 50] * 12, 8, 2, 64, 32), ([300, 0] * 40, [33, 5] * 40, 4, 2, 128, 128),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("case", TREES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", "")[:60])
def test_tree_attention(q3, case, dtype):
    import torch
    c = tree_case(np.random.default_rng(7), *case, dtype=getattr(torch, dtype))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_tree(q3, c, status=status)
    check_tree(c, out)
    assert int(status) == 0


@pytest.mark.parametrize("seqs,longest,most,heads,kv_heads,hd,page", [
    (97, 700, 13, 16, 8, 128, 16), (60, 1500, 1, 8, 8, 128, 16), (300, 90, 3, 4, 2, 64, 16),
    (70, 700, 9, 4, 1, 64, 8), (45, 600, 40, 8, 4, 128, 16), (41, 900, 16, 16, 8, 128, 12),
    (33, 800, 64, 2, 1, 64, 24), (60, 700, 64, 8, 4, 128, 16), (170, 300, 33, 8, 1, 64, 64)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_tree_attention_many_sequences(q3, dtype, seqs, longest, most, heads, kv_heads, hd, page):
    """More sequences, heads and row tiles than SMs: each SM works through several
    of them, one to many tiles long, some without nodes."""
    import torch
    rng = np.random.default_rng(8)
    lens, nodes = rng.integers(0, longest, seqs).tolist(), rng.integers(0, most + 1, seqs).tolist()
    c = tree_case(rng, lens, nodes, heads, kv_heads, hd, page, getattr(torch, dtype))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_tree(q3, c, status=status)
    check_tree(c, out)
    assert int(status) == 0 and torch.equal(out, run_tree(q3, c))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("heads,kv_heads,page,nodes", [(1024, 1, 16, 3), (999, 1, 16, 2), (14, 2, 12, 33), (27, 3, 16, 64)])
def test_many_and_odd_heads_to_a_kv_head(q3, heads, kv_heads, page, nodes, dtype):
    """Rows of one node in several tiles, tiles of rows of several nodes; rows before the
    first sequence's are left alone."""
    import torch
    c = tree_case(np.random.default_rng(22), [40, 0, 200], [nodes, 1, nodes // 2], heads, kv_heads, 64, page, getattr(torch, dtype))
    want = run_tree(q3, c)
    check_tree(c, want)
    q, m = torch.zeros((len(c["masks"]) + 5, heads, 64), device="cuda"), bu.masks_tensor([0] * 5 + c["masks"])
    q[5:] = c["q"]
    out = torch.full_like(q, -7.5)
    q3.tree_attention(c["pool"], 1, c["table"], c["lengths"], c["start"] + 5, m, q, max_nodes=nodes, out=out)
    assert torch.equal(out[5:], want) and bool((out[:5] == -7.5).all())


@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (600, 100)])
def test_chain_and_masks_that_see_nothing(q3, heads, kv_heads):
    """A chain is causal attention; a mask of zeroes sees the context only, and
    without a context nothing: zeroes, whatever the cache holds."""
    import torch
    c = tree_case(np.random.default_rng(9), [40, 0, 0], [12, 4, 5], heads, kv_heads, 128, 16, torch.bfloat16,
                  parents=[list(range(-1, 11)), [-1, 0, 1, 2], [-1] * 5])
    c["masks"][12 + 2] = 0
    c["masks"][3] = 0
    out = run_tree(q3, c)
    check_tree(c, out)
    assert bool((out[12 + 2] == 0).all())


@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (1920, 160)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_large_scores_and_masked_infinities(q3, dtype, heads, kv_heads):
    """Scores hundreds apart, rising along the context; infinities and NaN at
    nodes that no mask shows."""
    import torch
    c = tree_case(np.random.default_rng(10), [400], [6], heads, kv_heads, 128, 16, getattr(torch, dtype),
                  parents=[[-1, 0, -1, 2, -1, 4]])
    pos = torch.arange(406, device="cuda")
    pg, slot = c["table"][0].long()[pos // 16], pos % 16
    ramp = torch.linspace(0.02, 6.0, 406, device="cuda")[:, None, None, None]
    k = c["pool"][:, pg, 0, :, slot]
    c["pool"][:, pg, 0, :, slot] = (k.float() * ramp).to(k.dtype)
    for j, bad in ((404, math.inf), (405, math.nan)):  # nodes 4 and 5
        c["pool"][:, pg[j], :, :, slot[j]] = bad
    c["nodes"], c["masks"] = [6], c["masks"][:4] + [1, 2]
    out = run_tree(q3, c)
    c["pool"][:, pg[404], :, :, slot[404]] = 0
    c["pool"][:, pg[405], :, :, slot[405]] = 0
    # an unseen value still meets a weight of zero: only the keys may be infinite
    finite = torch.isfinite(out)
    want, tol = bu.tree_reference(c["pool"], 1, c["table"], c["lens"], c["nodes"], c["masks"], c["q"])
    assert bool(finite.all())
    assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("seqs,nodes", [(1, 3), (160, 64)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_scores_up_to_their_limit(q3, dtype, seqs, nodes):
    """Scores of 2^26 and 2^27, exact and of one sign in each head: the positions at the
    largest share the weight equally.  (Bound: some 20 roundings of a weight's sum and 16
    of an output's, 2^-24 each.)"""
    import torch
    n, hd = 300, 64
    c = tree_case(np.random.default_rng(23), [n] * seqs, [nodes] * seqs, 2, 1, hd, 16, getattr(torch, dtype))
    pos = torch.arange(n + nodes, device="cuda")
    small = (pos % 7 == 2) & (pos < n)  # at 2^26, the others at 2^27
    k = torch.zeros((n + nodes, hd), device="cuda")
    k[:, 0] = torch.where(small, -(2.0 ** 14), -(2.0 ** 15))
    c["q"][:] = 0
    c["q"][:, 0, 0], c["q"][:, 1, 0] = 2.0 ** 15, -(2.0 ** 15)
    for s in range(seqs):
        c["pool"][:, c["table"][s].long()[pos // 16], 0, 0, pos % 16] = k.to(c["pool"].dtype)
    out = run_tree(q3, c)
    for s in {0, seqs - 1}:
        v = c["pool"][1, c["table"][s].long()[pos // 16], 1, 0, pos % 16].double()
        for i in range(s * nodes, (s + 1) * nodes):
            sees = torch.tensor([j < n or bool(c["masks"][i] >> (j - n) & 1) for j in range(n + nodes)], device="cuda")
            for h, rows in ((0, small), (1, ~small & sees)):
                assert bool(((out[i, h].double() - v[rows].mean(0)).abs() <= 2.0 ** -18 * v[rows].abs().mean(0)).all())


@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (800, 80)])
def test_row_pitches_and_rows_left_alone(q3, heads, kv_heads):
    """q inside a wider buffer at an odd pitch, out likewise; rows behind the last
    sequence and other columns keep their values."""
    import torch
    c = tree_case(np.random.default_rng(11), [33, 90], [5, 7], heads, kv_heads, 64, 16, torch.bfloat16)
    wide = torch.full((15, heads * 64 + 37), 3.25, device="cuda")
    wide[:12, 1:heads * 64 + 1] = c["q"].reshape(12, -1)
    qv = wide[:, 1:heads * 64 + 1].unflatten(1, (heads, 64))
    outw = torch.full((15, heads * 64 + 3), -7.5, device="cuda")
    ov = outw[:, 3:].unflatten(1, (heads, 64))
    masks = torch.cat([bu.masks_tensor(c["masks"]), torch.zeros(3, dtype=torch.int64, device="cuda")])
    q3.tree_attention(c["pool"], 1, c["table"], c["lengths"], c["start"], masks, qv, max_nodes=7, out=ov)
    check_tree(c, ov[:12])
    assert bool((outw[12:] == -7.5).all()) and bool((outw[:, :3] == -7.5).all())


def test_queries_and_outputs_in_one_buffer(q3):
    """Outputs beside the queries of their rows; on them they are refused."""
    import torch
    c = tree_case(np.random.default_rng(20), [33, 90], [5, 7], 4, 2, 64, 16, torch.bfloat16)
    both = torch.zeros((12, 2, 4, 64), device="cuda")
    both[:, 0] = c["q"]
    c["q"] = both[:, 0]
    run_tree(q3, c, out=both[:, 1])
    check_tree(c, both[:, 1])
    for out in (both[:, 0], both.view(24, 4, 64)[1:13]):
        with pytest.raises(q3.Q3TTSError) as err:
            run_tree(q3, c, out=out)
        assert err.value.code == q3.ERR_ARG


@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (1440, 60)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_bad_device_entries_are_reported(q3, dtype, heads, kv_heads):
    """Lengths, row offsets and page ids that do not fit: reported, the others'
    rows are right, and the left-out rows keep their values."""
    import torch
    c = tree_case(np.random.default_rng(12), [20, 30, 40], [3, 3, 3], heads, kv_heads, 64, 16, getattr(torch, dtype))
    for change in ("length", "negative", "start", "page"):
        lengths, start, table = c["lengths"].clone(), c["start"].clone(), c["table"].clone()
        if change == "length":
            lengths[1] = table.shape[1] * 16 - 2
        elif change == "negative":
            lengths[1] = -1
        elif change == "start":
            start[3] = 100
        else:
            table[1, 1] = c["pool"].shape[1]
        out = torch.full_like(c["q"], -7.5)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q3.tree_attention(c["pool"], 1, table, lengths, start, bu.masks_tensor(c["masks"]), c["q"], max_nodes=3,
                          out=out, status=status)
        assert int(status) == q3.ERR_ARG
        want, tol = bu.tree_reference(c["pool"], 1, c["table"], c["lens"], c["nodes"], c["masks"], c["q"])
        bad = slice(6, 9) if change == "start" else slice(3, 6)
        ok = (out.double() - want).abs() <= tol
        ok[bad] = True
        assert bool(ok.all())
        if change != "page":
            assert bool((out[bad] == -7.5).all())


@pytest.mark.parametrize("heads,kv_heads", [(16, 8), (800, 100)])
def test_tree_attention_repeats_captures_and_follows_new_lengths(q3, heads, kv_heads):
    """The same bits on every run; a captured call replays with other lengths and
    masks; two graphs of it replay side by side on two streams."""
    import torch
    c = tree_case(np.random.default_rng(13), [250, 61], [9, 4], heads, kv_heads, 128, 16, torch.bfloat16)
    masks = bu.masks_tensor(c["masks"])
    first = run_tree(q3, c)
    assert torch.equal(first, run_tree(q3, c))
    outs = [torch.zeros_like(first) for _ in range(2)]
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for o, s in zip(outs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            q3.tree_attention(c["pool"], 1, c["table"], c["lengths"], c["start"], masks, c["q"], max_nodes=9, out=o)
        graphs.append(g)
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            for _ in range(5):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)
    c["lens"] = [100, 60]
    c["lengths"].copy_(torch.tensor(c["lens"], dtype=torch.int32))
    c["masks"] = bu.tree_masks([-1] * 9) + bu.tree_masks([-1, 0, 1, 2])
    masks.copy_(bu.masks_tensor(c["masks"]))
    graphs[0].replay()
    torch.cuda.synchronize()
    check_tree(c, outs[0])


def test_two_threads_at_once(q3):
    """Two host threads, each with its stream and tensors, many calls each."""
    import threading

    import torch
    rng = np.random.default_rng(17)
    jobs, errors = [], []
    for heads, kv_heads, seqs in ((16, 8, 3), (32, 4, 40)):
        c = tree_case(rng, rng.integers(0, 600, seqs).tolist(), rng.integers(0, 30, seqs).tolist(), heads, kv_heads, 128, 16,
                      torch.bfloat16)
        c["mask_rows"] = bu.masks_tensor(c["masks"])
        logits, scores = torch.randn((4, heads, 5000), device="cuda"), torch.zeros((4, heads), device="cuda")
        jobs.append((c, logits, scores, run_tree(q3, c), q3.beam_select(logits, scores)))
    torch.cuda.synchronize()

    def work(c, logits, scores, want, picks):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    out = q3.tree_attention(c["pool"], 1, c["table"], c["lengths"], c["start"], c["mask_rows"], c["q"],
                                            max_nodes=max(c["nodes"]))
                    got = q3.beam_select(logits, scores)
                    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(got, picks))
        except BaseException as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


LOST = [
    # lens, nodes, heads, kv heads, head dim, page: an SM's one short item, an item shared by a
    # cluster, several items of several tiles to an SM
    ([131], [8], 2, 1, 128, 16), ([9000], [8], 2, 1, 128, 16), ([600] * 200, [8] * 200, 2, 1, 128, 16),
    ([131], [16], 2, 1, 64, 16), ([9000], [16], 4, 2, 64, 16), ([600] * 200, [16] * 200, 2, 1, 128, 16),
    ([131], [32], 2, 1, 128, 16), ([9000], [32], 2, 1, 128, 16), ([600] * 200, [32] * 200, 2, 1, 64, 16),
    # more than 64 rows to a kv head
    ([600] * 160, [64] * 160, 2, 1, 128, 16), ([600] * 160, [64] * 160, 2, 1, 64, 16), ([9000], [64], 38, 19, 128, 16),
    # pages that boxes do not fit
    ([131], [8], 2, 1, 128, 12), ([9000], [16], 2, 1, 128, 12), ([600] * 200, [32] * 200, 2, 1, 64, 12)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("tile", [0, 1, 3])
@pytest.mark.parametrize("case", LOST, ids=lambda c: "-".join(str(x) for x in c).replace(" ", "")[:20] + "-" + "-".join(
    str(x) for x in (c[1][0], *c[2:])))
def test_a_wait_that_runs_out(q3, case, tile, dtype):
    """The products of one CTA never come: its waits run out after 2 ms, the call
    reports it, and the next one is right (copies and tensor memory given back)."""
    import time

    import torch
    c = tree_case(np.random.default_rng(18), *case, dtype=getattr(torch, dtype))
    masks = bu.masks_tensor(c["masks"])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run():
        status.zero_()
        out = q3.tree_attention(c["pool"], 1, c["table"], c["lengths"], c["start"], masks, c["q"],
                                max_nodes=max(c["nodes"]), status=status)
        return out, int(status)

    want, code = run()
    assert code == 0
    q3.debug_lose_tile(1 << 30, 2000000)  # no such tile
    out, code = run()
    assert code == 0 and torch.equal(out, want)
    for _ in range(2):
        q3.debug_lose_tile(tile, 2000)
        t0 = time.perf_counter()
        code = run()[1]
        if tile < -(-(case[0][0] + case[1][0]) // 128):
            assert code == q3.ERR_TIMEOUT and time.perf_counter() - t0 < 1.0
        else:
            assert code == 0
        out, code = run()
        assert code == 0 and torch.equal(out, want)


FIRST_CALLS = """
import torch
from autoregressive_tts_decode_gb300 import q3tts
from tests import branch_util as bu
import numpy as np
rng = np.random.default_rng(15)
pool, table = bu.paged_cache(rng, [1030] * 8, 16, 2, 8, 128, torch.bfloat16)
i32 = dict(dtype=torch.int32, device="cuda")
lengths, start = torch.full((8,), 1000, **i32), torch.arange(9, **i32) * 30
masks = bu.masks_tensor(sum((bu.tree_masks(bu.tree_parents(rng, 30)) for _ in range(8)), []))
q = torch.randn((240, 32, 128), device="cuda")
logits, scores = torch.randn((2, 4, 9000), device="cuda"), torch.zeros((2, 4), device="cuda")
path, count = torch.tensor([[1, 3]] * 8, **i32), torch.full((8,), 2, **i32)
torch.cuda.synchronize()
kept = pool.clone()

def calls():
    out = q3tts.tree_attention(pool, 1, table, lengths, start, masks, q, max_nodes=30)
    few = q3tts.tree_attention(pool, 0, table, lengths, start, masks, q[:, :8].contiguous(), max_nodes=30)
    picks = q3tts.beam_select(logits, scores)
    moved = torch.empty_like(logits)
    q3tts.reorder_rows([logits], [moved], picks[1])
    q3tts.copy_pages(pool, [0], [pool.shape[1] - 1])
    q3tts.compact_rows(pool, table, lengths, path, count)
    return out, few, *picks, moved

g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = calls()
bits = lambda x: x.view(torch.int16)  # (unused places hold NaN)
assert torch.equal(bits(pool), bits(kept))  # nothing ran yet
g.replay()
torch.cuda.synchronize()
after, got = pool.clone(), [x.clone() for x in got]
pool.copy_(kept)
for a, b in zip(got, calls()):
    assert torch.equal(a, b)
assert torch.equal(bits(after), bits(pool))
print("same")
"""


def test_first_calls_inside_a_capture():
    """A process whose first call of each operator is a captured one."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


FIRST_THREADS = """
import threading, torch
from autoregressive_tts_decode_gb300 import q3tts
from tests import branch_util as bu
import numpy as np
rng = np.random.default_rng(19)
pool, table = bu.paged_cache(rng, [300] * 4, 16, 2, 8, 128, torch.bfloat16)
i32 = dict(dtype=torch.int32, device="cuda")
lengths, start = torch.full((4,), 290, **i32), torch.arange(5, **i32) * 10
masks = bu.masks_tensor(sum((bu.tree_masks(bu.tree_parents(rng, 10)) for _ in range(4)), []))
q = torch.randn((40, 16, 128), device="cuda")
jobs = [(torch.randn(s, device="cuda"), torch.zeros(s[:2], device="cuda")) for s in ((2, 4, 900), (1, 9, 20000)) * 4]
torch.cuda.synchronize()
gate, got, errors = threading.Barrier(8), [None] * 8, []

def calls(logits, scores):
    picks = q3tts.beam_select(logits, scores)
    moved = torch.empty_like(logits)
    q3tts.reorder_rows([logits], [moved], picks[1])
    return [q3tts.tree_attention(pool, 1, table, lengths, start, masks, q, max_nodes=10), *picks, moved]

def work(i):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            gate.wait()
            got[i] = calls(*jobs[i])
            torch.cuda.current_stream().synchronize()
    except BaseException as e:
        errors.append(e)

threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not errors, errors
for g, j in zip(got, jobs):
    assert all(torch.equal(a, b) for a, b in zip(g, calls(*j)))
print("same")
"""


def test_first_calls_of_many_threads():
    """A process whose first calls are eight threads' at once."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_THREADS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_cache_offsets_past_32_bits(q3):
    """A cache of more than 2^32 elements: pages near its end are read and copied."""
    import torch
    pages = 70000
    pool = torch.zeros((1, pages, 2, 4, 64, 128), dtype=torch.bfloat16, device="cuda")  # 4.6e9 elements, 9.2 GB
    rng = np.random.default_rng(14)
    gen = torch.Generator(device="cuda").manual_seed(3)
    used = [pages - 1, pages - 5, 2]
    for p in used:
        pool[0, p] = torch.randn((2, 4, 64, 128), generator=gen, device="cuda").to(torch.bfloat16)
    lens, nodes = [150], [20]
    masks = bu.tree_masks(bu.tree_parents(rng, 20))
    table = torch.tensor([used], dtype=torch.int32, device="cuda")
    q = torch.randn((20, 4, 128), generator=gen, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    out = q3.tree_attention(pool, 0, table, torch.tensor(lens, **i32), torch.tensor([0, 20], **i32),
                            bu.masks_tensor(masks), q, max_nodes=20)
    want, tol = bu.tree_reference(pool, 0, table, lens, nodes, masks, q)
    assert bool(((out.double() - want).abs() <= tol).all())
    q3.copy_pages(pool, [pages - 1], [pages - 2])
    assert torch.equal(pool[0, pages - 1], pool[0, pages - 2])


# ------------------------------------------------------------------ pages
@pytest.mark.parametrize("n", [1, 3, 449])
@pytest.mark.parametrize("shape", [(2, 1, 16, 64), (3, 2, 12, 128), (1, 8, 16, 128), (5, 1, 1, 64)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_copy_pages(q3, n, shape, dtype):
    import torch
    layers, heads, page, hd = shape
    pages = 2 * n + 3
    pool = torch.randn((layers, pages, 2, heads, page, hd), device="cuda").to(getattr(torch, dtype))
    want = pool.clone()
    perm = np.random.default_rng(n).permutation(pages)[:2 * n]
    src = perm[:n].tolist()
    src[0] = src[-1]  # one page may be copied to several
    want[:, perm[n:].tolist()] = want[:, src]
    q3.copy_pages(pool, src, perm[n:].tolist())
    assert torch.equal(pool, want)


@pytest.mark.parametrize("page,hd,dtype", [(16, 128, "bfloat16"), (12, 64, "float32"), (1, 64, "bfloat16"),
                                           (64, 128, "float32")])
def test_compact_rows(q3, page, hd, dtype):
    import torch
    rng = np.random.default_rng(page)
    lens, most = [0, 5, 31, 64, 100, 7], 64
    pool, table = bu.paged_cache(rng, [n + most for n in lens], page, 3, 2, hd, getattr(torch, dtype))
    paths = [list(range(64)), [], [0, 1, 5, 6, 63], sorted(rng.permutation(64)[:40].tolist()), [63],
             list(range(1, 64))]
    path = np.full((len(lens), most), -9, np.int32)
    for s, p in enumerate(paths):
        path[s, :len(p)] = p
    want = pool.clone()
    for s, p in enumerate(paths):
        for to, of in enumerate(p):
            a, b = lens[s] + of, lens[s] + to
            want[:, table[s, b // page], :, :, b % page] = pool[:, table[s, a // page], :, :, a % page]
    i32 = dict(dtype=torch.int32, device="cuda")
    status = torch.zeros(1, **i32)
    q3.compact_rows(pool, table, torch.tensor(lens, **i32), torch.from_numpy(path).cuda(),
                    torch.tensor([len(p) for p in paths], **i32), status=status)
    assert torch.equal(torch.nan_to_num(pool.float()), torch.nan_to_num(want.float())) and int(status) == 0


@pytest.mark.parametrize("page,hd,dtype", [(16, 128, "bfloat16"), (7, 64, "float32")])
def test_compact_rows_of_long_paths(q3, page, hd, dtype):
    """Paths of more rows than a CTA looks up at a time."""
    import torch
    rng = np.random.default_rng(31)
    lens, most = [13, 0, 100], 700
    pool, table = bu.paged_cache(rng, [n + most for n in lens], page, 2, 3, hd, getattr(torch, dtype))
    paths = [sorted(rng.permutation(most)[:513].tolist()), list(range(1, most)), sorted(rng.permutation(most)[:256].tolist())]
    path = np.zeros((3, most), np.int32)
    want = pool.clone()
    for s, p in enumerate(paths):
        path[s, :len(p)] = p
        to, of = (torch.tensor(x, device="cuda") + lens[s] for x in (list(range(len(p))), p))
        tb = table[s].long()
        want[:, tb[to // page], :, :, to % page] = pool[:, tb[of // page], :, :, of % page]
    i32 = dict(dtype=torch.int32, device="cuda")
    status = torch.zeros(1, **i32)
    q3.compact_rows(pool, table, torch.tensor(lens, **i32), torch.from_numpy(path).cuda(),
                    torch.tensor([len(p) for p in paths], **i32), status=status)
    assert torch.equal(torch.nan_to_num(pool.float()), torch.nan_to_num(want.float())) and int(status) == 0


@pytest.mark.parametrize("bad", ["descending", "twice", "negative", "long", "count", "length"])
def test_compact_rows_leaves_bad_sequences(q3, bad):
    import torch
    rng = np.random.default_rng(5)
    pool, table = bu.paged_cache(rng, [40, 40], 16, 2, 2, 64, torch.bfloat16)
    before = pool.clone()
    i32 = dict(dtype=torch.int32, device="cuda")
    path = {"descending": [3, 2, 5], "twice": [2, 2, 5], "negative": [-1, 2, 5], "long": [1, 2, 40]}.get(bad, [1, 2, 5])
    lengths, count = [30, 30], [3, 3]
    if bad == "count":
        count[0] = 4
    if bad == "length":
        lengths[0] = -1
    status = torch.zeros(1, **i32)
    q3.compact_rows(pool, table, torch.tensor(lengths, **i32), torch.tensor([path, [1, 2, 5]], **i32),
                    torch.tensor(count, **i32), status=status)
    assert int(status) == q3.ERR_ARG
    seq0 = table[0].long()
    seq0 = seq0[seq0 < pool.shape[1]]
    assert torch.equal(torch.nan_to_num(pool[:, seq0].float()), torch.nan_to_num(before[:, seq0].float()))
    a, b = 31, 30
    assert torch.equal(pool[:, table[1, b // 16], :, :, b % 16], before[:, table[1, a // 16], :, :, a % 16])


# ------------------------------------------------------------------ beams
def run_beam(q3, logits, scores, k, **kw):
    import torch
    for n in ("history", "finished"):
        if kw.get(n) is not None:
            kw[n] = torch.from_numpy(kw[n]).cuda()
    return [t.cpu().numpy() for t in q3.beam_select(torch.from_numpy(logits).cuda(), torch.from_numpy(scores).cuda(),
                                                    k=k, **kw)]


def check_beam(got, logits, scores, k, history=None, finished=None, eos_token=-1, special_from=0,
               repetition_penalty=1.0):
    """The scores' order decides; candidates closer than the fp32 sums can tell
    (each exponential and sum within a few 2^-24 of the row's sum: 2^-20 covers
    vocabularies up to 2^17 summed in fp32 by 512 threads) may swap."""
    kw = dict(history=history, finished=finished, eos=eos_token, special=special_from, penalty=repetition_penalty)
    tok, par, best = bu.beam_reference(logits, scores, k, **kw)
    sc, _ = bu.beam_scores(logits, scores, **kw)
    gt, gp, gs = got
    live = best > -np.inf
    assert np.array_equal(gt == -1, ~live) and np.all(gp[~live] == 0) and np.all(np.isneginf(gs[~live]))
    eps = 2.0 ** -20
    assert np.all(np.abs(gs[live] - best[live]) <= eps + 2.0 ** -24 * np.abs(best[live]))
    for g, j in zip(*np.nonzero(live)):
        assert abs(sc[g, gp[g, j], gt[g, j]] - best[g, j]) <= eps
    for g in range(gt.shape[0]):
        pairs = [(int(a), int(b)) for a, b, ok in zip(gp[g], gt[g], live[g]) if ok]
        assert len(set(pairs)) == len(pairs)
    return np.array_equal(gt, tok) and np.array_equal(gp, par)


@pytest.mark.parametrize("groups,beams,k,vocab", [(1, 1, 1, 1), (1, 1, 4, 7), (3, 4, 4, 2048), (2, 5, 3, 4095),
                                                  (1, 32, 32, 4096), (2, 3, 32, 33), (1, 1, 8, 100003),
                                                  (2, 2, 5, 32768), (5, 16, 16, 8193), (1, 2, 32, 9)])
def test_beam_select(q3, groups, beams, k, vocab):
    rng = np.random.default_rng(vocab + k)
    logits = (3 * rng.standard_normal((groups, beams, vocab))).astype(np.float32)
    scores = (-5 * rng.random((groups, beams))).astype(np.float32)
    assert check_beam(run_beam(q3, logits, scores, k), logits, scores, k)


def test_beam_workspace(q3):
    """Groups of up to eight rows that are scanned whole need none; others are
    refused with too little."""
    import torch
    rng = np.random.default_rng(16)
    for groups, beams, vocab in ((1, 4, 2048), (2, 8, 8192), (3, 9, 2048), (1, 4, 100003)):
        logits, scores = rng.standard_normal((groups, beams, vocab)).astype(np.float32), np.zeros((groups, beams), np.float32)
        need = q3.beam_workspace_size(groups, beams, vocab, beams)
        assert (need == 0) == (beams <= 8 and vocab <= 8192)
        args = torch.from_numpy(logits).cuda(), torch.from_numpy(scores).cuda()
        got = q3.beam_select(*args, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
        for a, b in zip(got, q3.beam_select(*args)):
            assert torch.equal(a, b)
        if need:
            with pytest.raises(q3.Q3TTSError) as err:
                q3.beam_select(*args, workspace=torch.empty(need - 8, dtype=torch.uint8, device="cuda"))
            assert err.value.code == q3.ERR_ARG


@pytest.mark.parametrize("vocab", [50, 2048, 20001])
def test_beam_select_rules(q3, vocab):
    """Penalty, special codes, finished beams, dead beams."""
    rng = np.random.default_rng(vocab)
    g, b, k = 4, 6, 6
    logits = (2 * rng.standard_normal((g, b, vocab))).astype(np.float32)
    scores = (-5 * rng.random((g, b))).astype(np.float32)
    scores[1, 2:] = -np.inf
    scores[2, 0] = np.nan
    kw = dict(history=(rng.random((g, b, vocab)) < 0.3).astype(np.uint8),
              finished=(rng.random((g, b)) < 0.4).astype(np.uint8), eos_token=vocab - 3, special_from=vocab - 20,
              repetition_penalty=1.3)
    kw["finished"][3] = 1
    assert check_beam(run_beam(q3, logits, scores, k, **dict(kw)), logits, scores, k, **kw)


@pytest.mark.parametrize("vocab", [6, 2048, 8192, 40000])
@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "masked", "infinite", "nan", "huge"])
def test_beam_select_hard_rows(q3, kind, vocab):
    """Equal logits (the lower code, the lower beam first), sorted ones, rows with
    little or nothing to pick, infinities and NaN."""
    g, b, k = 2, 3, 8
    rng = np.random.default_rng(vocab)
    logits = np.zeros((g, b, vocab), np.float32)
    scores = np.zeros((g, b), np.float32)
    if kind == "ascending":
        logits += np.arange(vocab, dtype=np.float32) / 64
    elif kind == "descending":
        logits -= np.arange(vocab, dtype=np.float32) / 64
    elif kind == "masked":
        logits[:] = -np.inf
        logits[0, 1, vocab // 2] = 1.5
        logits[0, 2, [0, vocab - 1]] = -3e38
    elif kind == "infinite":
        logits = rng.standard_normal((g, b, vocab)).astype(np.float32)
        logits[0, 0, [1, 4]] = np.inf
        logits[1, :, 3] = np.inf
        logits[1, 1, 0] = -np.inf
    elif kind == "nan":
        logits = rng.standard_normal((g, b, vocab)).astype(np.float32)
        logits[0, 0, ::2] = np.nan
        logits[1, 1] = np.nan
    elif kind == "huge":
        logits = (1e38 * rng.standard_normal((g, b, vocab)).clip(-3, 3)).astype(np.float32)
    assert check_beam(run_beam(q3, logits, scores, k), logits, scores, k)


@pytest.mark.parametrize("vocab", [2, 600, 8192, 20001])
def test_beam_select_signed_zeros_are_equal(q3, vocab):
    """-0 and +0 are equal logits: the lower code first, within a tile and across."""
    logits = np.zeros((1, 2, vocab), np.float32)
    logits[0, :, ::2] = -0.0
    logits[0, 1, vocab // 3:] = 0.0
    logits[0, 1, :vocab // 3] = -0.0
    scores = np.zeros((1, 2), np.float32)
    k = min(vocab, 7)
    tok, par, _ = run_beam(q3, logits, scores, k)
    assert tok.tolist() == [list(range(k))] and (par == 0).all()
    tok, par, _ = run_beam(q3, logits[:, 1:], scores[:, 1:], k)
    assert tok.tolist() == [list(range(k))]


@pytest.mark.parametrize("vocab", [9, 2048, 20001])
def test_beam_select_infinite_and_huge_scores(q3, vocab):
    """A beam at +infinity stays there (its best logits first), one at -infinity or NaN
    has no candidate; scores at the end of fp32's range keep their order."""
    rng = np.random.default_rng(vocab)
    logits = (2 * rng.standard_normal((4, 4, vocab))).astype(np.float32)
    logits[2, 1, vocab // 2] = np.inf
    big = np.float32(3.4028234e38)
    scores = np.array([[0, np.inf, -np.inf, 1], [np.nan, -np.inf, -np.inf, -np.inf], [1, np.inf, -1, np.inf],
                       [-big, big, -big, 2e37]], np.float32)
    got = run_beam(q3, logits, scores, 6)
    tok, par, best = bu.beam_reference(logits, scores, 6)
    assert np.array_equal(got[2], best.astype(np.float32))
    assert np.array_equal(got[1], par) and np.array_equal(got[0], tok)


def test_beam_select_row_ids_pitch_and_in_place_scores(q3):
    import torch
    rng = np.random.default_rng(21)
    rows, vocab = 11, 1001
    full = (2 * rng.standard_normal((rows, vocab + 6))).astype(np.float32)
    hist = (rng.random((rows, vocab)) < 0.2).astype(np.uint8)
    fin = (rng.random(rows) < 0.3).astype(np.uint8)
    ids = rng.permutation(rows)[:6].reshape(2, 3).astype(np.int32)
    scores = (-rng.random((2, 3))).astype(np.float32)
    lg = torch.from_numpy(full).cuda()[:, 3:3 + vocab]
    sc = torch.from_numpy(scores).cuda()
    out = (torch.zeros((2, 3), dtype=torch.int32, device="cuda"), torch.zeros((2, 3), dtype=torch.int32, device="cuda"),
           sc)
    kw = dict(eos_token=5, repetition_penalty=1.2)
    q3.beam_select(lg, sc, row_ids=torch.from_numpy(ids).cuda(), history=torch.from_numpy(hist).cuda(),
                   finished=torch.from_numpy(fin).cuda(), out=out, **kw)
    assert check_beam([t.cpu().numpy() for t in out], full[ids][..., 3:3 + vocab], scores, 3, history=hist[ids],
                      finished=fin[ids], **kw)


@pytest.mark.parametrize("tail,dtype", [((64,), "float32"), ((7,), "uint8"), ((3, 5), "float32"), ((), "uint8"),
                                        ((2000,), "bfloat16"), ((4099,), "int64")])
@pytest.mark.parametrize("groups,beams,k", [(1, 1, 1), (3, 4, 4), (2, 3, 7), (1, 32, 32), (2, 9, 2)])
def test_reorder_rows(q3, tail, dtype, groups, beams, k):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(1)
    src = torch.randint(0, 200, (groups, beams) + tail, generator=gen, device="cuda").to(getattr(torch, dtype))
    par = torch.randint(0, beams, (groups, k), generator=gen, device="cuda").int()
    want = torch.stack([src[g, par[g].long()] for g in range(groups)])
    dst = torch.empty_like(want)
    q3.reorder_rows([src], [dst], par)
    assert torch.equal(dst, want)
    if beams == k:
        sets = [src.clone() for _ in range(9)]  # more sets than one launch takes
        q3.reorder_rows(sets, sets, par)
        assert all(torch.equal(t, want) for t in sets)


def test_reorder_rows_reports_bad_parents(q3):
    import torch
    for inplace in (False, True):
        src = torch.arange(12, device="cuda", dtype=torch.float32).reshape(1, 3, 4).clone()
        dst = src if inplace else torch.full_like(src, -1)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        par = torch.tensor([[2, 3, 0]], dtype=torch.int32, device="cuda")
        want = [8.0, 4.0 if inplace else -1.0, 0.0]
        q3.reorder_rows([src], [dst], par, status=status)
        assert int(status) == q3.ERR_ARG and dst[0, :, 0].tolist() == want


def test_reorder_rows_refuses_buffers_exchanged(q3):
    import torch
    a, b = torch.randn((1, 3, 4), device="cuda"), torch.randn((1, 3, 4), device="cuda")
    par = torch.tensor([[2, 2, 0]], dtype=torch.int32, device="cuda")
    for src, dst in (([a, b], [b, a]), ([a, a], [a, a]), ([a, b], [b, b]), ([par], [par])):
        with pytest.raises(q3.Q3TTSError) as err:
            q3.reorder_rows(src, dst, par)
        assert err.value.code == q3.ERR_ARG
    out = torch.empty((2, 1, 3, 4), device="cuda")
    q3.reorder_rows([a, a], [out[0], out[1]], par)  # one source may be read twice
    assert torch.equal(out[0], a[:, [2, 2, 0]]) and torch.equal(out[1], out[0])


def test_reorder_rows_of_records_with_fields(q3):
    """Rows that lie between each other's: two fields of a record in place, and a
    third into a fourth."""
    import ctypes as C

    import torch
    rec = torch.arange(6 * 64, device="cuda", dtype=torch.uint8).reshape(6, 64)
    par = torch.tensor([[1, 1, 0], [2, 0, 0]], dtype=torch.int32, device="cuda")
    want, rows = rec.clone(), torch.tensor([1, 1, 0, 5, 3, 3], device="cuda")
    want[:, 0:16], want[:, 20:27], want[:, 48:64] = rec[rows, 0:16], rec[rows, 20:27], rec[rows, 32:48]
    p = rec.data_ptr()
    sets = (q3.Rows * 3)(q3.Rows(p, p, 16, 64, 64), q3.Rows(p + 20, p + 20, 7, 64, 64), q3.Rows(p + 32, p + 48, 16, 64, 64))
    s = torch.cuda.current_stream().cuda_stream
    assert q3.load().q3tts_reorder_rows(sets, 3, None, par.data_ptr(), 2, 3, 3, None, s) == q3.OK
    assert torch.equal(rec, want)


# --------------------------------------------------------------- together
def test_a_search_step_with_the_operators(q3):
    """Trees are scored for two sequences, paths accepted, a page forked, beams
    selected and their states moved: each step reads what the one before wrote,
    on a stream other than the default, and captured into a graph."""
    import torch
    rng = np.random.default_rng(30)
    c = tree_case(rng, [37, 90], [6, 6], 8, 4, 128, 16, torch.bfloat16,
                  parents=[[-1, 0, 0, 1, 3, 2], [-1, -1, 1, 2, 2, 4]])
    paths = [[0, 2, 5], [1, 2, 4]]
    i32 = dict(dtype=torch.int32, device="cuda")
    path, count = torch.tensor(paths, **i32), torch.tensor([3, 3], **i32)
    after = c["lengths"] + count
    one = torch.tensor([0, 1, 2], **i32)
    bit = torch.zeros(2, dtype=torch.int64, device="cuda")
    spare = [p for p in range(c["pool"].shape[1]) if p not in c["table"].flatten().tolist()]
    last = int(c["table"][0, 39 // 16])
    q2 = torch.randn((2, 8, 128), device="cuda")
    logits, scores = torch.randn((1, 2, 500), device="cuda"), torch.zeros((1, 2), device="cuda")
    state, moved = torch.randn((1, 2, 65), device="cuda"), torch.empty((1, 2, 65), device="cuda")
    before = c["pool"].clone()
    res = {}

    def step():
        res["tree"] = run_tree(q3, c)
        q3.compact_rows(c["pool"], c["table"], c["lengths"], path, count)
        res["next"] = q3.tree_attention(c["pool"], 1, c["table"], after, one, bit, q2, max_nodes=1)
        q3.copy_pages(c["pool"], [last], [spare[0]])
        res["beam"] = q3.beam_select(logits, scores)
        q3.reorder_rows([state], [moved], res["beam"][1])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for captured in (False, True):
        c["pool"].copy_(before)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            if captured:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=s):
                    res["tree"] = q3.tree_attention(c["pool"], 1, c["table"], c["lengths"], c["start"], res["m"],
                                                    c["q"], max_nodes=6)
                    q3.compact_rows(c["pool"], c["table"], c["lengths"], path, count)
                    res["next"] = q3.tree_attention(c["pool"], 1, c["table"], after, one, bit, q2, max_nodes=1)
                    q3.copy_pages(c["pool"], [last], [spare[0]])
                    res["beam"] = q3.beam_select(logits, scores)
                    q3.reorder_rows([state], [moved], res["beam"][1])
                g.replay()
            else:
                res["m"] = bu.masks_tensor(c["masks"])
                step()
        torch.cuda.synchronize()
        kept, c["pool"] = c["pool"], before
        check_tree(c, res["tree"])
        c["pool"] = kept
        # the accepted nodes' rows now follow the context, and the node that
        # attends to the context alone sees them
        for i, p in enumerate(paths):
            for to, of in enumerate(p):
                a, b = c["lens"][i] + of, c["lens"][i] + to
                assert torch.equal(c["pool"][:, c["table"][i, b // 16], :, :, b % 16],
                                   before[:, c["table"][i, a // 16], :, :, a % 16])
        full = torch.nan_to_num(c["pool"])
        want, tol = bu.tree_reference(full, 1, c["table"], after.tolist(), [1, 1], [0, 0], q2)
        assert bool(((res["next"].double() - want).abs() <= tol).all())
        assert torch.equal(torch.nan_to_num(c["pool"][:, spare[0]].float()), torch.nan_to_num(c["pool"][:, last].float()))
        tok, par, best = (t.cpu().numpy() for t in res["beam"])
        assert check_beam([tok, par, best], logits.cpu().numpy(), scores.cpu().numpy(), 2)
        assert torch.equal(moved, state[:, par[0].tolist()])
