"""Branching decode on a handle: forks, trees of drafted frames and beam frames
against streams that were prefilled and stepped one by one."""
import ctypes as C
import dataclasses
import math

import numpy as np
import pytest

from autoregressive_tts_decode_gb300 import synth
from tests import branch_util as bu
from tests import parity_util as pu

pytestmark = pytest.mark.gpu

TINY = synth.TINY_SHAPE
GREEDY = synth.GREEDY
SAMPLED = synth.QWEN_DEFAULT_SAMPLING


@pytest.fixture(scope="module")
def q3():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from autoregressive_tts_decode_gb300 import build, q3tts
    build.build()
    return q3tts


@pytest.fixture(scope="module")
def weights():
    return {"f32": pu.gpu_weights(TINY)[1],
            "bf16": pu.gpu_weights(dataclasses.replace(TINY, weight_dtype=synth.DTYPE_BF16))[1]}


SHAPES = {
    "f32": TINY,
    "bf16": dataclasses.replace(TINY, weight_dtype=synth.DTYPE_BF16, kv_dtype=synth.DTYPE_BF16),
}
# The same positions computed by other launches (other batch widths, other
# splits): fp32 sums in another order.  With a bf16 cache a key or value may
# round to its neighbour (a relative 2^-8 of one element).
TOL = {"f32": 2e-4, "bf16": 2e-2}


def engine(q3, weights, kind, streams, cap=128, page=16, **kw):
    return q3.Engine(SHAPES[kind], weights[kind], streams, cap, page_size=page, **kw)


def prompt(n, seed=1):
    return synth.make_prompts(TINY, [n], seed=seed)[0].cuda()


def frame(eng, ids, sp, f, forced=None, streams_for_uniforms=None, logits=None):
    import torch
    u = torch.from_numpy(np.ascontiguousarray(synth.uniforms(streams_for_uniforms or [0] * len(ids), 40)[:, f])).cuda()
    c = torch.zeros((len(ids), 16), dtype=torch.int32, device="cuda")
    fc = None if forced is None else torch.from_numpy(np.ascontiguousarray(forced, dtype=np.int32)).cuda()
    eng.step_frame(ids, sp, u, c, forced=fc, logits=logits)
    eng.sync()
    return c.cpu().numpy()


def frame_like(a, b, ids, sp, f, history, orc, tol, streams_for_uniforms=None):
    """One frame of both handles, b fed with a's codes: the logits of all 16 draws
    agree, and each handle's codes are the sampler's on its own logits with the
    given histories, exactly.  The codes themselves are not compared: a frame sums
    in an order that changes from run to run, so the logits of two runs of one and
    the same frame differ in their last bits, and a uniform within that of a
    boundary between two codes draws either (prompt of 45, no path, frame 1,
    codebook 13: 23 of 800 runs of step_frame drew the other one)."""
    import torch
    Vt, Vc = TINY.codec_vocab, TINY.cp_vocab
    us = streams_for_uniforms or [0] * len(ids)
    u = synth.uniforms(us, 40)[:, f]
    out, fed = [], None
    for e in (a, b):
        lg = torch.zeros((len(ids), Vt + 15 * Vc), dtype=torch.float32, device="cuda")
        c = frame(e, ids, sp, f, forced=fed, streams_for_uniforms=us, logits=lg)
        out.append(lg.cpu().numpy())
        fed = c if fed is None else fed
        for r, s in enumerate(ids):
            hist = np.zeros(Vt, dtype=np.uint8)
            hist[history[s]] = 1
            lr = out[-1][r]
            want = [orc.sample(lr[:Vt], sp.do_sample, sp.top_k, sp.top_p, sp.temperature, sp.repetition_penalty,
                               hist, float(u[r, 0]), special_from=getattr(sp, "special_from", 0),
                               eos_token=getattr(sp, "eos_token", -1))]
            want += [orc.sample(lr[Vt + j * Vc:Vt + (j + 1) * Vc], sp.sub_do_sample, sp.sub_top_k, sp.sub_top_p,
                                sp.sub_temperature, 1.0, None, float(u[r, j + 1])) for j in range(15)]
            assert c[r].tolist() == want
    assert np.max(np.abs(out[0] - out[1])) <= tol
    for r, s in enumerate(ids):
        history[s].append(int(fed[r, 0]))
    return fed


def random_codes(rng, n):
    return np.concatenate([rng.integers(0, TINY.codec_vocab, (n, 1)), rng.integers(0, TINY.cp_vocab, (n, 15))],
                          axis=1).astype(np.int32)


def pending(eng, sid):
    h, lg = eng.read_pending(sid)
    eng.sync()
    return h.cpu().numpy(), lg.cpu().numpy()


# ------------------------------------------------------------------- fork
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("plen,page", [(16, 16), (21, 16), (30, 12)])
def test_forked_streams_go_on_like_their_source(q3, weights, oracle_mod, kind, plen, page):
    """Prompt, two frames, fork into two more (one of which held another stream):
    all three decode the same codes as a handle with three separate prompts."""
    a = engine(q3, weights, kind, 4, page=page)
    b = engine(q3, weights, kind, 4, page=page)
    a.prefill(1, prompt(plen))
    a.prefill(3, prompt(50, seed=9))
    for s in (1, 3, 0):
        b.prefill(s, prompt(plen))
    past = []
    for f in range(2):
        forced = frame(a, [1], SAMPLED, f)
        past.append(int(forced[0, 0]))
        frame(b, [1], SAMPLED, f, forced=forced)
        frame(b, [3, 0], SAMPLED, f, forced=np.repeat(forced, 2, 0))
    a.fork(1, [3, 0])
    assert [a.length(s) for s in (0, 1, 3)] == [plen + 2] * 3
    for s in (3, 0):
        for x, y in zip(pending(a, s), pending(a, 1)):
            assert np.array_equal(x, y)
    history = {s: list(past) for s in (1, 3, 0)}
    for f in range(2, 6):
        # the takes part ways: other uniforms for each
        frame_like(a, b, [1, 3, 0], SAMPLED, f, history, oracle_mod, TOL[kind], [5, 6, 7])
        for s in (1, 3, 0):
            assert np.max(np.abs(pending(a, s)[1] - pending(b, s)[1])) <= TOL[kind]
    a.close(), b.close()


def test_forks_share_pages_and_give_them_back(q3, weights):
    """12 pages hold a prompt of 9.x pages and two takes of it, which separate
    prompts could not; a take that ends frees its own pages only."""
    eng = engine(q3, weights, "f32", 4, cap=192, kv_pages=12)
    eng.prefill(0, prompt(150))
    with pytest.raises(q3.Q3TTSError) as e:
        eng.prefill(1, prompt(150))
    assert e.value.code == q3.ERR_CAPACITY
    eng.fork(0, [1, 2])  # 10 pages, and two copies of the last
    with pytest.raises(q3.Q3TTSError) as e:
        eng.fork(0, [3])
    assert e.value.code == q3.ERR_CAPACITY and eng.length(3) == 0
    # a target's own page counts as room: forking into it again works
    eng.fork(0, [2])
    want = frame(eng, [0, 1, 2], GREEDY, 0)
    assert np.array_equal(want[0], want[1]) and np.array_equal(want[0], want[2])
    eng.reset(0)  # the source may end first
    frame(eng, [1, 2], GREEDY, 1)
    eng.reset(1)
    eng.prefill(3, prompt(20, seed=4))  # the freed copies
    assert eng.length(2) == 152
    eng.reset()
    eng.prefill(0, prompt(180))  # the whole pool again
    eng.close()


def test_fork_into_many_streams(q3, weights):
    eng = engine(q3, weights, "f32", 40, cap=64)
    eng.prefill(7, prompt(18))
    dst = [s for s in range(40) if s != 7]
    eng.fork(7, dst)
    c = frame(eng, list(range(40)), GREEDY, 0)
    assert (c == c[0]).all()
    eng.close()


def test_branch_calls_refuse(q3, weights):
    import torch
    eng = engine(q3, weights, "f32", 4, cap=32)
    codes = torch.zeros((64, 16), dtype=torch.int32, device="cuda")

    def code(f):
        with pytest.raises(q3.Q3TTSError) as e:
            f()
        return e.value.code

    assert code(lambda: eng.fork(0, [1])) == q3.ERR_STATE
    assert code(lambda: eng.tree_step(0, codes, [-1])) == q3.ERR_STATE
    eng.prefill(0, prompt(20))
    for src, dst in ((0, []), (0, [0]), (0, [1, 1]), (0, [4]), (0, [-1]), (4, [1]), (-1, [1])):
        assert code(lambda: eng.fork(src, dst)) == q3.ERR_ARG
    for parents in ([], [0], [-1, 1], [-2], [-1] * 65):
        assert code(lambda: eng.tree_step(0, torch.zeros((80, 16), dtype=torch.int32, device="cuda"), parents)) == q3.ERR_ARG
    assert code(lambda: eng.tree_step(0, codes, [-1] * 13)) == q3.ERR_CAPACITY
    assert code(lambda: eng.tree_accept(0, [0])) == q3.ERR_STATE
    eng.tree_step(0, codes, [-1, 0, 0, -1])
    for path in ([4], [-1], [1], [0, 3], [0, 1, 2], [3, 0]):
        assert code(lambda: eng.tree_accept(0, path)) == q3.ERR_ARG
    assert code(lambda: eng.tree_accept(1, [0])) == q3.ERR_STATE
    frame(eng, [0], GREEDY, 0)  # the stream moved on: its tree is gone
    assert code(lambda: eng.tree_accept(0, [0])) == q3.ERR_STATE
    u = torch.zeros((4, 16), device="cuda")
    sc = torch.zeros((2, 2), device="cuda")
    cc = torch.zeros((4, 16), dtype=torch.int32, device="cuda")
    assert code(lambda: eng.beam_frame([[0, 1]], GREEDY, sc, u, cc)) == q3.ERR_STATE
    eng.fork(0, [1, 2, 3])
    for ids in ([[0, 0]], [[0, 4]], [[0, -1]], [[0, 1, 2, 3], [0, 1, 2, 3]]):
        assert code(lambda: eng.beam_frame(ids, GREEDY, torch.zeros(8, device="cuda"),
                                           torch.zeros((8, 16), device="cuda"),
                                           torch.zeros((8, 16), dtype=torch.int32, device="cuda"))) == q3.ERR_ARG
    assert eng.length(0) == 21
    # codes outside their vocabulary are reported, and the handle goes on
    bad = codes.clone()
    bad[0, 3] = TINY.cp_vocab
    eng.tree_step(0, bad, [-1])
    assert code(eng.sync) == q3.ERR_ARG
    eng.tree_accept(0, [])
    frame(eng, [0], GREEDY, 1)
    assert eng.length(0) == 22
    eng.close()


# ------------------------------------------------------------------- trees
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("plen,page,parents", [
    (16, 16, [-1, 0, 1, 2, 3]),                               # a chain
    (29, 16, [-1, 0, 0, 1, -1, 4, 5, 2, 6]),                  # branches, over a page's end
    (21, 12, [-1] + [0] * 9 + [3, 10, 11, 12, 13, 5, 15]),
    (3, 16, [-1] * 5)])
def test_tree_nodes_equal_forced_frames(q3, weights, kind, plen, page, parents):
    """Each node's hidden and logits are what a fork of the stream has after the
    node's path was fed frame by frame."""
    import torch
    rng = np.random.default_rng(len(parents))
    n = len(parents)
    codes = random_codes(rng, n)
    eng = engine(q3, weights, kind, 3, page=page)
    eng.prefill(0, prompt(plen))
    hid = torch.zeros((n, TINY.talker_hidden), device="cuda")
    lg = torch.zeros((n, TINY.codec_vocab), device="cuda")
    eng.tree_step(0, torch.from_numpy(codes).cuda(), parents, hidden=hid, logits=lg)
    eng.sync()
    assert eng.length(0) == plen
    for i in range(n):
        path, j = [], i
        while j >= 0:
            path.insert(0, j)
            j = parents[j]
        eng.fork(0, [1])
        for d, j in enumerate(path):
            frame(eng, [1], GREEDY, d, forced=codes[j:j + 1])
        h, l = pending(eng, 1)
        assert np.max(np.abs(h - hid[i].cpu().numpy())) <= TOL[kind] * 5
        assert np.max(np.abs(l - lg[i].cpu().numpy())) <= TOL[kind]
    eng.close()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("path", [[], [0], [0, 1, 3], [4, 5], [0, 2]])
def test_accepted_path_becomes_the_context(q3, weights, oracle_mod, kind, path):
    """After accepting a path the stream decodes on as one that was fed the same
    frames, with the same history; unused pages are back in the pool."""
    import torch
    parents = [-1, 0, 0, 1, -1, 4] + [5] * 30
    codes = random_codes(np.random.default_rng(3), len(parents))
    a = engine(q3, weights, kind, 1, kv_pages=6, cap=96)
    b = engine(q3, weights, kind, 1, kv_pages=6, cap=96)
    for e in (a, b):
        e.prefill(0, prompt(45))
    a.tree_step(0, torch.from_numpy(codes).cuda(), parents)
    a.tree_accept(0, path)
    for j in path:
        frame(b, [0], GREEDY, 0, forced=codes[j:j + 1])
    assert a.length(0) == b.length(0) == 45 + len(path)
    sp = dataclasses.replace(SAMPLED, repetition_penalty=1.5)
    history = {0: codes[path, 0].tolist()}
    for f in range(1, 5):
        frame_like(a, b, [0], sp, f, history, oracle_mod, TOL[kind])
        assert np.max(np.abs(pending(a, 0)[1] - pending(b, 0)[1])) <= TOL[kind]
    a.close(), b.close()


@pytest.mark.parametrize("then", ["frame", "static", "fork", "beam", "prefill", "reset", "tree"])
def test_a_tree_that_no_path_is_taken_of(q3, weights, then):
    """A drafted tree leaves its stream as it was for whatever comes next, and is
    gone once that call has changed the stream."""
    import torch
    parents = [-1] + [0] * 39
    codes = torch.from_numpy(random_codes(np.random.default_rng(4), len(parents))).cuda()
    a, b = (engine(q3, weights, "f32", 2, cap=96) for _ in range(2))
    for e in (a, b):
        e.prefill(0, prompt(41))
        e.prefill(1, prompt(30, seed=2))
    a.tree_step(0, codes, parents)
    for e in (a, b):
        u, c = torch.full((1, 16), 0.5, device="cuda"), torch.zeros((1, 16), dtype=torch.int32, device="cuda")
        if then == "frame":
            frame(e, [0], GREEDY, 0)
        elif then == "static":
            e.step_frame_static(0, GREEDY, u, c)
        elif then == "fork":
            e.fork(0, [1])
        elif then == "beam":
            e.beam_frame([[0, 1]], GREEDY, torch.tensor([[0.0, -math.inf]], device="cuda"), u.repeat(2, 1), c.repeat(2, 1))
        elif then == "prefill":
            e.prefill(0, prompt(20, seed=5))
        elif then == "reset":
            e.reset(0)
            e.prefill(0, prompt(33, seed=6))
        else:
            hid = torch.zeros((3, TINY.talker_hidden), device="cuda")
            e.tree_step(0, codes[5:8].contiguous(), [-1, 0, 1], hidden=hid)
            e.tree_accept(0, [0, 1])
        e.sync()
    if then != "fork":
        with pytest.raises(q3.Q3TTSError) as err:
            a.tree_accept(0, [0])
        assert err.value.code == q3.ERR_STATE
    for f in range(1, 3):
        for s in (0, 1):
            frame(a, [s], GREEDY, f, forced=frame(b, [s], GREEDY, f))
            assert a.length(s) == b.length(s)
            for x, y in zip(pending(a, s), pending(b, s)):
                assert np.max(np.abs(x - y)) <= TOL["f32"] * 5
    a.close(), b.close()


@pytest.mark.parametrize("plen", [30, 32])
def test_other_calls_between_a_tree_and_its_acceptance(q3, weights, plen):
    """Forks of the tree's stream, frames, beams, prompts and trees that are refused leave
    the tree; the forks are not touched when it is accepted."""
    import torch
    parents = [-1, 0, 0, 1, -1, 4] + [5] * 20
    codes = random_codes(np.random.default_rng(6), len(parents))
    dev = torch.from_numpy(codes).cuda()
    path = [0, 2]
    a, b = engine(q3, weights, "f32", 5, cap=80), engine(q3, weights, "f32", 5, cap=80)
    for e in (a, b):
        e.prefill(0, prompt(plen))
        e.prefill(1, prompt(20, seed=2))
        e.prefill(2, prompt(20, seed=2))
    a.tree_step(0, dev, parents)
    a.fork(0, [3])
    frame(a, [1, 3], GREEDY, 0, forced=codes[7:9])
    a.beam_frame([[1, 2]], GREEDY, torch.zeros((1, 2), device="cuda"), torch.zeros((2, 16), device="cuda"),
                 torch.zeros((2, 16), dtype=torch.int32, device="cuda"))
    a.prefill(4, prompt(33, seed=5))
    with pytest.raises(q3.Q3TTSError):
        a.tree_step(1, torch.zeros((64, 16), dtype=torch.int32, device="cuda"), [-1] * 64)
    a.tree_accept(0, path)
    for j in path:
        frame(b, [0], GREEDY, 0, forced=codes[j:j + 1])
    b.prefill(3, prompt(plen))
    frame(b, [3], GREEDY, 0, forced=codes[8:9])
    for f in range(1, 3):
        for s in (0, 3):
            frame(b, [s], GREEDY, f, forced=frame(a, [s], GREEDY, f))
            assert a.length(s) == b.length(s)
            for x, y in zip(pending(a, s), pending(b, s)):
                assert np.max(np.abs(x - y)) <= TOL["f32"] * 5
    a.close(), b.close()


@pytest.mark.parametrize("then", ["frame", "static", "frames of both", "tree", "smaller tree", "fork", "beam"])
def test_a_dropped_tree_gives_its_pages_back(q3, weights, then):
    """A tree of 40 frames fills the pool; whatever drops it returns its pages, so
    that another stream's prompt fits, and the refused calls before leave it."""
    import torch
    parents = [-1] + [0] * 39
    codes = torch.from_numpy(random_codes(np.random.default_rng(4), 64)).cuda()
    eng = engine(q3, weights, "f32", 3, cap=96, kv_pages=7)
    eng.prefill(0, prompt(41))             # 3 pages
    eng.prefill(1, prompt(16, seed=2))     # 1 page, full
    eng.tree_step(0, codes, parents)       # 3 more
    u, c = torch.full((2, 16), 0.5, device="cuda"), torch.zeros((2, 16), dtype=torch.int32, device="cuda")

    def full(f):
        with pytest.raises(q3.Q3TTSError) as e:
            f()
        assert e.value.code == q3.ERR_CAPACITY

    full(lambda: frame(eng, [1], GREEDY, 0))                                    # opens a page
    full(lambda: eng.tree_step(1, codes, [-1] * 64))                            # 4 more pages: one too many
    eng.tree_accept(0, []) if then == "fork" else None                          # (a fork leaves its source's tree)
    if then == "frame":
        frame(eng, [0], GREEDY, 0)
    elif then == "static":
        eng.step_frame_static(0, GREEDY, u, c)
    elif then == "frames of both":
        frame(eng, [0, 1], GREEDY, 0)      # the tree's pages are the other's new one
        assert eng.length(1) == 17
    elif then == "tree":
        eng.tree_step(1, codes, [-1] * 40)  # 3 pages: the first tree's
        eng.tree_accept(1, [])
    elif then == "smaller tree":
        eng.tree_step(0, codes, [-1, 0])
        eng.prefill(2, prompt(48, seed=3))
        eng.reset(2)
        eng.tree_accept(0, [0, 1])
        assert eng.length(0) == 43
    elif then == "fork":
        eng.fork(0, [2])
        eng.reset(2)
    else:
        eng.beam_frame([[0]], GREEDY, torch.zeros((1, 1), device="cuda"), u[:1].contiguous(), c[:1].contiguous())
    left = 7 - 3 - (2 if then == "frames of both" else 1)
    full(lambda: eng.prefill(2, prompt(16 * left + 1, seed=3)))
    eng.prefill(2, prompt(16 * left, seed=3))
    want = engine(q3, weights, "f32", 3, cap=96)
    want.prefill(2, prompt(16 * left, seed=3))
    for x, y in zip(pending(eng, 2), pending(want, 2)):
        assert np.max(np.abs(x - y)) <= TOL["f32"] * 5
    eng.close(), want.close()


# ------------------------------------------------------------------- beams
def test_one_beam_is_the_greedy_decode(q3, weights):
    import torch
    sp = dataclasses.replace(GREEDY, repetition_penalty=1.3)
    a, b = engine(q3, weights, "f32", 2), engine(q3, weights, "f32", 2)
    for e in (a, b):
        for s in range(2):
            e.prefill(s, prompt(20, seed=s))
    sc = torch.zeros((2, 1), device="cuda")
    c = torch.zeros((2, 16), dtype=torch.int32, device="cuda")
    u = torch.zeros((2, 16), device="cuda")
    for f in range(5):
        par = a.beam_frame([[0], [1]], sp, sc, u, c)
        assert (par == 0).all()
        want = frame(b, [0, 1], sp, f)
        assert np.array_equal(c.cpu().numpy(), want)
    assert bool((sc < 0).all())
    a.close(), b.close()


@pytest.mark.parametrize("kind,page,stop", [("f32", 16, False), ("f32", 12, True), ("bf16", 16, True)])
def test_beam_frames_equal_a_plain_search(q3, weights, kind, page, stop):
    """Two groups of three beams: every frame's selection is the 64-bit one of
    the pending logits, and every beam's state is that of a stream fed its whole
    history of codes from the prompt."""
    import torch
    groups, beams, frames = 2, 3, 7
    eng = engine(q3, weights, kind, 6, page=page)
    ref = engine(q3, weights, kind, 6, page=page)
    sp = dataclasses.replace(GREEDY, repetition_penalty=1.2)
    if stop:
        sp = dataclasses.replace(sp, special_from=TINY.codec_vocab - 40, eos_token=TINY.codec_vocab - 7)
    ids = [[4, 0, 2], [1, 5, 3]]
    plens = [30, 13]
    for g in range(groups):
        eng.prefill(ids[g][0], prompt(plens[g], seed=g))
        eng.fork(ids[g][0], ids[g][1:])
        for b in range(beams):
            ref.prefill(ids[g][b], prompt(plens[g], seed=g))
    scores = np.array([[0, -np.inf, -np.inf]] * 2, np.float32)
    sc = torch.from_numpy(scores).cuda()
    c = torch.zeros((6, 16), dtype=torch.int32, device="cuda")
    u = torch.zeros((6, 16), device="cuda")
    fed = [[[] for _ in range(beams)] for _ in range(groups)]  # each beam's frames so far
    done = np.zeros((groups, beams), np.uint8)
    for f in range(frames):
        lg = np.stack([[pending(eng, s)[1] for s in row] for row in ids])
        hist = np.zeros((groups, beams, TINY.codec_vocab), np.uint8)
        for g in range(groups):
            for b in range(beams):
                for x in fed[g][b]:
                    hist[g, b, x[0]] = 1
        kw = dict(history=hist, special=sp.special_from, eos=sp.eos_token, penalty=sp.repetition_penalty)
        if stop:
            kw["finished"] = done
        tok, par, best = bu.beam_reference(lg, scores, beams, **kw)
        got_par = eng.beam_frame(ids, sp, sc, u, c)
        eng.sync()
        codes = c.cpu().numpy().reshape(groups, beams, 16)
        scores = sc.cpu().numpy()
        live = best > -np.inf
        assert np.array_equal(got_par, par)
        assert np.max(np.abs(scores[live] - best[live])) <= 1e-4
        new = [[list(fed[g][par[g, b]]) for b in range(beams)] for g in range(groups)]
        nd = np.zeros_like(done)
        for g in range(groups):
            for b in range(beams):
                was = done[g, par[g, b]]
                if was:
                    assert (codes[g, b] == -1).all()
                else:
                    assert codes[g, b, 0] == tok[g, b]
                    new[g][b].append(codes[g, b])
                nd[g, b] = was or (stop and tok[g, b] == sp.eos_token)
        fed, done = new, nd
    # every live beam against a stream that was fed its frames one by one
    for g in range(groups):
        for b in range(beams):
            if done[g, b]:
                continue
            s = ids[g][b]
            for f, x in enumerate(fed[g][b]):
                frame(ref, [s], GREEDY, f, forced=x[None])
            assert ref.length(s) == eng.length(s)
            assert np.max(np.abs(pending(eng, s)[1] - pending(ref, s)[1])) <= TOL[kind]
    assert len({tuple(x[0] for x in fed[0][b]) for b in range(beams)}) == beams
    eng.close(), ref.close()


@pytest.mark.parametrize("beams,extra", [(4, 2), (8, 2), (9, 3)])
def test_beam_frame_counts_its_launches(q3, weights, beams, extra):
    """A frame of as many streams, and the selection (one launch up to eight beams, two
    beyond) and the reordering; the context ends with a page, so none is copied."""
    import torch
    eng = engine(q3, weights, "f32", beams)
    eng.prefill(0, prompt(16))
    eng.fork(0, list(range(1, beams)))
    u = torch.full((beams, 16), 0.5, device="cuda")
    c = torch.zeros((beams, 16), dtype=torch.int32, device="cuda")
    sc = torch.tensor([[0.0] + [-math.inf] * (beams - 1)], device="cuda")
    counts = [eng.kernel_launches()]
    eng.beam_frame([list(range(beams))], GREEDY, sc, u, c)
    counts.append(eng.kernel_launches())
    eng.step_frame(list(range(beams)), GREEDY, u, c)
    counts.append(eng.kernel_launches())
    eng.sync()
    assert counts[1] - counts[0] == counts[2] - counts[1] + extra
    eng.close()


def test_a_finished_beam_keeps_its_score(q3, weights):
    """A group whose beams have all fed the end code stays as it is."""
    import torch
    v = TINY.codec_vocab
    sp = dataclasses.replace(GREEDY, special_from=1, eos_token=v - 1)  # codes 0 and the end code
    eng = engine(q3, weights, "f32", 2)
    eng.prefill(0, prompt(20))
    eng.fork(0, [1])
    sc = torch.tensor([[0.0, -np.inf]], device="cuda")
    c = torch.zeros((2, 16), dtype=torch.int32, device="cuda")
    u = torch.zeros((2, 16), device="cuda")
    for _ in range(12):
        eng.beam_frame([[0, 1]], sp, sc, u, c)
    eng.sync()
    codes, scores = c.cpu().numpy(), sc.cpu().numpy()
    assert scores[0, 0] >= scores[0, 1] and np.isfinite(scores).all()
    assert eng.finished(0) or eng.finished(1)
    for b in range(2):
        assert (codes[b] == -1).all() == eng.finished(b) or codes[b, 0] in (0, v - 1)
    eng.close()


def test_beam_frame_without_room_changes_nothing(q3, weights):
    import torch
    eng = engine(q3, weights, "f32", 3, cap=64, kv_pages=3)
    eng.prefill(0, prompt(32))  # two whole pages, shared; each beam opens one of its own
    eng.fork(0, [1, 2])
    sc = torch.tensor([[0.0, -np.inf, -np.inf]], device="cuda")
    c = torch.zeros((3, 16), dtype=torch.int32, device="cuda")
    u = torch.zeros((3, 16), device="cuda")
    before = [pending(eng, s) for s in range(3)]
    with pytest.raises(q3.Q3TTSError) as e:
        eng.beam_frame([[0, 1, 2]], GREEDY, sc, u, c)
    assert e.value.code == q3.ERR_CAPACITY
    assert sc.cpu().tolist() == [[0.0, -np.inf, -np.inf]] and [eng.length(s) for s in range(3)] == [32] * 3
    for s in range(3):
        assert all(np.array_equal(x, y) for x, y in zip(pending(eng, s), before[s]))
    eng.reset(2), eng.reset(1)
    eng.beam_frame([[0]], GREEDY, sc[:, :1].contiguous(), u, c)
    assert eng.length(0) == 33
    eng.close()


def test_other_streams_are_left_alone(q3, weights):
    """Forks, trees and beams of some streams between the frames of another."""
    import torch
    a, b = engine(q3, weights, "f32", 5), engine(q3, weights, "f32", 5)
    for e in (a, b):
        e.prefill(4, prompt(17, seed=8))
    a.prefill(0, prompt(22))
    sc = torch.tensor([[0.0, -np.inf]], device="cuda")
    c = torch.zeros((2, 16), dtype=torch.int32, device="cuda")
    u = torch.zeros((2, 16), device="cuda")
    codes = torch.from_numpy(random_codes(np.random.default_rng(1), 6)).cuda()
    for f in range(4):
        a.fork(0, [1])
        a.tree_step(0, codes, [-1, 0, 0, 1, 2, -1])
        a.beam_frame([[0, 1]], SAMPLED, sc, u, c)
        a.tree_step(1, codes, [-1, 0, 0, 1, 2, -1])
        a.tree_accept(1, [0, 2])
        a.fork(1, [0, 2])
        a.reset(2)
        assert np.array_equal(frame(a, [4], SAMPLED, f), frame(b, [4], SAMPLED, f))
    a.close(), b.close()


def test_another_stream_between_branches_draws_its_own_codes(q3, weights, oracle_mod):
    """The same as above, compared as frame_like compares: the other stream's logits
    agree and its codes are the sampler's on its own logits."""
    import torch
    a, b = engine(q3, weights, "f32", 5), engine(q3, weights, "f32", 5)
    for e in (a, b):
        e.prefill(4, prompt(17, seed=8))
    a.prefill(0, prompt(22))
    sc = torch.tensor([[0.0, -np.inf]], device="cuda")
    c = torch.zeros((2, 16), dtype=torch.int32, device="cuda")
    u = torch.zeros((2, 16), device="cuda")
    codes = torch.from_numpy(random_codes(np.random.default_rng(1), 6)).cuda()
    history = {4: []}
    for f in range(4):
        a.fork(0, [1])
        a.tree_step(0, codes, [-1, 0, 0, 1, 2, -1])
        a.beam_frame([[0, 1]], SAMPLED, sc, u, c)
        a.tree_step(1, codes, [-1, 0, 0, 1, 2, -1])
        a.tree_accept(1, [0, 2])
        a.fork(1, [0, 2])
        a.reset(2)
        frame_like(a, b, [4], SAMPLED, f, history, oracle_mod, TOL["f32"])
    a.close(), b.close()


def test_a_finished_beams_score_stays_its_own(q3, weights):
    """Of two codes one is the end code, so that a beam ends in the first frame: from
    then on a slot whose parent has ended has the parent's score, bit for bit, feeds
    nothing and stays ended."""
    import torch
    v = TINY.codec_vocab
    sp = dataclasses.replace(GREEDY, special_from=1, eos_token=v - 1)  # codes 0 and the end code
    beams = 3
    eng = engine(q3, weights, "f32", beams)
    eng.prefill(0, prompt(20))
    eng.fork(0, [1, 2])
    sc = torch.tensor([[0.0, -np.inf, -np.inf]], device="cuda")
    c = torch.zeros((beams, 16), dtype=torch.int32, device="cuda")
    u = torch.zeros((beams, 16), device="cuda")
    stayed = 0
    for f in range(8):
        before, ended = sc.cpu().numpy()[0], [eng.finished(s) for s in range(beams)]
        par = eng.beam_frame([[0, 1, 2]], sp, sc, u, c)[0]
        eng.sync()
        after, codes = sc.cpu().numpy()[0], c.cpu().numpy()
        for b in range(beams):
            if ended[par[b]] and after[b] > -np.inf:
                stayed += 1
                assert after[b] == before[par[b]] and (codes[b] == -1).all() and eng.finished(b)
            elif after[b] > -np.inf:
                assert after[b] < before[par[b]] and codes[b, 0] in (0, v - 1)
                assert eng.finished(b) == (codes[b, 0] == v - 1)
        if f == 0:  # both codes, and no third continuation
            assert sorted(codes[:2, 0].tolist()) == [0, v - 1] and after[2] == -np.inf
    assert stayed >= 8
    eng.close()
