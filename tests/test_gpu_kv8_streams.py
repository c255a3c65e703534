"""The 8-bit cache's attention beside other calls on other streams, whose CTAs share SMs, shared
and tensor memory with its own: every result is that of a call alone."""
import numpy as np
import pytest

from tests import branch_util as bu
from tests import kv8_util as ku
from tests import test_gpu_kv8 as t8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from autoregressive_tts_decode_gb300 import build, q3tts
    build.build()
    return q3tts


def kv8_call(q3, rng, lens, rows, heads, kvh, hd, tree):
    c = t8.attend_case(rng, lens, rows, heads, kvh, hd, 16, 16, "bfloat16", tree)
    pool, scales, tab = ku.to_gpu(c["codes"], c["powers"], c["table"])
    m = bu.masks_tensor(c["masks"]) if tree else None
    args = pool, scales, 1, tab, ku.ints(lens), ku.ints(ku.starts(rows)), c["q"]
    return lambda: q3.kv8_attention(*args, masks=m, max_rows=max(rows))


def tree_call(q3, rng, lens, rows, heads, kvh, hd, dtype):
    import torch
    pool, table = bu.paged_cache(rng, [a + b for a, b in zip(lens, rows)], 16, 1, kvh, hd, dtype)
    masks = bu.masks_tensor(sum((bu.tree_masks(bu.tree_parents(rng, n)) for n in rows), []))
    q = t8.randn(rng, (sum(rows), heads, hd), torch.float32)
    args = pool, 0, table, ku.ints(lens), ku.ints(ku.starts(rows)), masks, q
    return lambda: q3.tree_attention(*args, max_nodes=max(rows))


@pytest.mark.parametrize("seqs", [1, 9])
def test_calls_on_three_streams(q3, seqs):
    """Single tokens, drafted trees and chunks over 8-bit caches beside tree attentions of 32 rows over bf16 and
    fp32 caches, all of them split over clusters, in turns and without waiting."""
    import torch
    rng = np.random.default_rng(71)
    calls = [[kv8_call(q3, rng, [3000] * seqs, [1] * seqs, 4, 2, 64, False), kv8_call(q3, rng, [900] * seqs, [7] * seqs, 4, 2, 64, True),
              kv8_call(q3, rng, [2500] * seqs, [64] * seqs, 4, 2, 128, True)],
             [tree_call(q3, rng, [2000] * seqs, [16] * seqs, 4, 2, 64, torch.bfloat16), tree_call(q3, rng, [1500] * seqs, [32] * seqs, 2, 2, 64, torch.float32)],
             [tree_call(q3, rng, [1000] * seqs, [5] * seqs, 4, 2, 64, torch.bfloat16), kv8_call(q3, rng, [700] * seqs, [300] * seqs, 2, 1, 64, False),
              kv8_call(q3, rng, [5000] * seqs, [1] * seqs, 2, 2, 64, False)]]
    want = [[f() for f in fs] for fs in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for turn in range(60):
        for fs, s, g in zip(calls, streams, got):
            with torch.cuda.stream(s):
                g.append(fs[turn % len(fs)]())
    torch.cuda.synchronize()
    for fs, w, g in zip(calls, want, got):
        assert all(torch.equal(x, w[i % len(fs)]) for i, x in enumerate(g))
