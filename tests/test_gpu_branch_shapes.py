"""Branching decode at a head dimension of 128, over contexts of several tiles of
positions and page sizes that tiles are and are not a multiple of, with each weight
and cache type: trees, accepted paths and beams against streams stepped one by one."""
import dataclasses
import math

import numpy as np
import pytest

from autoregressive_tts_decode_gb300 import synth
from tests import branch_util as bu
from tests import parity_util as pu

pytestmark = pytest.mark.gpu

BASE = dataclasses.replace(synth.TINY_SHAPE, n_q_heads=8, n_kv_heads=2, head_dim=128, codec_vocab=1500, cp_vocab=900)
KINDS = {
    "f32": dict(),
    "bf16": dict(weight_dtype=synth.DTYPE_BF16, kv_dtype=synth.DTYPE_BF16),
    "fp8": dict(weight_dtype=synth.DTYPE_FP8, kv_dtype=synth.DTYPE_BF16),
    "fp8 f32": dict(weight_dtype=synth.DTYPE_FP8),
}
# As for the tiny shape: fp32 sums in another order; with 16-bit activation terms or a
# bf16 cache an element may round to its neighbour (a relative 2^-8).
TOL = {"f32": 2e-4, "bf16": 2e-2, "fp8": 2e-2, "fp8 f32": 2e-2}


@pytest.fixture(scope="module")
def q3():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from autoregressive_tts_decode_gb300 import build, q3tts
    build.build()
    return q3tts


@pytest.fixture(scope="module")
def weights():
    made = {}

    def get(kind):
        s = dataclasses.replace(BASE, **KINDS[kind])
        if s.weight_dtype not in made:
            made[s.weight_dtype] = pu.gpu_weights(s)[1]
        return s, made[s.weight_dtype]

    return get


def engine(q3, weights, kind, streams, cap, page):
    s, w = weights(kind)
    return q3.Engine(s, w, streams, cap, page_size=page)


def prompt(n, seed=1):
    return synth.make_prompts(BASE, [n], seed=seed)[0].cuda()


def random_codes(rng, n):
    return np.concatenate([rng.integers(0, BASE.codec_vocab, (n, 1)), rng.integers(0, BASE.cp_vocab, (n, 15))],
                          axis=1).astype(np.int32)


def feed(eng, sid, code):
    import torch
    c = torch.zeros((1, 16), dtype=torch.int32, device="cuda")
    eng.step_frame([sid], synth.GREEDY, torch.zeros((1, 16), device="cuda"), c,
                   forced=torch.from_numpy(code[None].copy()).cuda())


def pending(eng, sid):
    h, lg = eng.read_pending(sid)
    eng.sync()
    return h.cpu().numpy(), lg.cpu().numpy()


def path_of(parents, i):
    out = []
    while i >= 0:
        out.insert(0, i)
        i = parents[i]
    return out


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("plen,page,n", [(300, 16, 30), (509, 24, 20), (250, 128, 64), (700, 16, 3)])
def test_trees_over_long_contexts(q3, weights, kind, plen, page, n):
    import torch
    rng = np.random.default_rng(n)
    parents = bu.tree_parents(rng, n)
    codes = random_codes(rng, n)
    eng = engine(q3, weights, kind, 2, plen + n + 4, page)
    eng.prefill(0, prompt(plen))
    hid = torch.zeros((n, BASE.talker_hidden), device="cuda")
    lg = torch.zeros((n, BASE.codec_vocab), device="cuda")
    eng.tree_step(0, torch.from_numpy(codes).cuda(), parents, hidden=hid, logits=lg)
    eng.sync()
    deepest = max(range(n), key=lambda i: len(path_of(parents, i)))
    for i in {0, n - 1, n // 2, deepest}:
        eng.fork(0, [1])
        for j in path_of(parents, i):
            feed(eng, 1, codes[j])
        h, l = pending(eng, 1)
        assert np.max(np.abs(h - hid[i].cpu().numpy())) <= TOL[kind] * 5
        assert np.max(np.abs(l - lg[i].cpu().numpy())) <= TOL[kind]
    # stream 1 was fed the deepest path last or is fed it now; stream 0 accepts it
    eng.fork(0, [1])
    path = path_of(parents, deepest)
    for j in path:
        feed(eng, 1, codes[j])
    eng.tree_accept(0, path)
    assert eng.length(0) == eng.length(1) == plen + len(path)
    more = random_codes(rng, 2)
    for code in more:
        for s in (0, 1):
            feed(eng, s, code)
        for x, y, f in zip(pending(eng, 0), pending(eng, 1), (5, 1)):
            assert np.max(np.abs(x - y)) <= TOL[kind] * f
    eng.close()


@pytest.mark.parametrize("kind", list(KINDS))
def test_beams_over_long_contexts(q3, weights, kind):
    """Every beam's state after some frames is that of a stream fed its codes."""
    import torch
    beams, frames, plen = 4, 5, 270
    eng, ref = (engine(q3, weights, kind, beams, plen + 16, 16) for _ in range(2))
    eng.prefill(0, prompt(plen))
    eng.fork(0, [1, 2, 3])
    sc = torch.tensor([[0.0] + [-math.inf] * 3], device="cuda")
    c = torch.zeros((beams, 16), dtype=torch.int32, device="cuda")
    u = torch.zeros((beams, 16), device="cuda")
    fed = [[] for _ in range(beams)]
    for _ in range(frames):
        lg = np.stack([pending(eng, s)[1] for s in range(beams)])[None]
        tok, par, best = bu.beam_reference(lg, sc.cpu().numpy(), beams)
        got = eng.beam_frame([[0, 1, 2, 3]], synth.GREEDY, sc, u, c)
        eng.sync()
        codes = c.cpu().numpy()
        assert np.array_equal(got, par) and np.array_equal(codes[None, :, 0], tok)
        assert np.max(np.abs(sc.cpu().numpy() - best)) <= 1e-4
        fed = [fed[p] + [codes[b].copy()] for b, p in enumerate(par[0])]
    for b in range(beams):
        ref.prefill(b, prompt(plen))
        for x in fed[b]:
            feed(ref, b, x)
        assert np.max(np.abs(pending(eng, b)[1] - pending(ref, b)[1])) <= TOL[kind]
    eng.close(), ref.close()
