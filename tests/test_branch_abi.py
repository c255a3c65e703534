"""Refusals of the branching-decode entries without a GPU: every argument check
answers before any device work (the pointers are made up and never followed)."""
import ctypes as C
import os
import re
from struct import calcsize

import numpy as np
import pytest

from autoregressive_tts_decode_gb300 import build, q3tts

A = 1 << 40  # a made-up device address


@pytest.fixture(scope="module")
def lib():
    build.build()
    return q3tts.load()


def cache(**kw):
    f = dict(pool=A, layers=2, n_pages=10, n_kv_heads=2, page_size=16, head_dim=64, kv_dtype=q3tts.BF16)
    f.update(kw)
    return q3tts.KVCache(*[f[n] for n, _ in q3tts.KVCache._fields_])


BAD_CACHES = [(dict(pool=None), q3tts.ERR_ARG), (dict(pool=A + 8), q3tts.ERR_ARG), (dict(layers=0), q3tts.ERR_ARG),
              (dict(n_pages=0), q3tts.ERR_ARG), (dict(n_kv_heads=0), q3tts.ERR_ARG),
              (dict(page_size=0), q3tts.ERR_ARG), (dict(kv_dtype=q3tts.FP8), q3tts.ERR_ARG),
              (dict(head_dim=96), q3tts.ERR_UNSUPPORTED)]


def header():
    return open(os.path.join(os.path.dirname(build.HERE), "include", "q3tts_branch.h")).read()


def test_exports_every_declared_function(lib):
    names = set(re.findall(r"^(?:int|size_t) (q3tts_[a-z_]+)\(", header(), re.M))
    assert names == set(q3tts.BRANCH_EXPORTS) and not names & set(q3tts.EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def test_struct_layouts_match_header():
    src = header()
    for name, struct in (("q3tts_kv_cache", q3tts.KVCache), ("q3tts_rows", q3tts.Rows)):
        body = re.search(r"typedef struct " + name + r" \{(.*?)\} " + name, src, re.S).group(1)
        names = [n.strip().split()[-1].lstrip("*") for d in body.split(";") if d.strip() for n in d.split(",")]
        assert names == [f[0] for f in struct._fields_]
    # the binding packs the same layouts as bytes
    assert q3tts._CACHE.size == C.sizeof(q3tts.KVCache) and calcsize(q3tts._ROWS) == C.sizeof(q3tts.Rows)
    consts = dict(re.findall(r"#define (Q3TTS_[A-Z_0-9]+) \(?(-?\d+)\)?", src))
    assert int(consts["Q3TTS_MAX_TREE_NODES"]) == q3tts.MAX_TREE_NODES
    assert int(consts["Q3TTS_MAX_BEAMS"]) == q3tts.MAX_BEAMS


TREE = ["layer", "table", "pps", "n_seqs", "lengths", "start", "masks", "n_rows", "max_nodes", "heads", "q", "ldq",
        "out", "ldo", "status"]


def tree(lib, kv=None, **kw):
    a = dict(layer=0, table=A, pps=4, n_seqs=2, lengths=A, start=A, masks=A, n_rows=8, max_nodes=4, heads=4, q=A,
             ldq=256, out=A + 65536, ldo=256, status=None)
    a.update(kw)
    return lib.q3tts_tree_attention(C.byref(kv or cache()), *[a[n] for n in TREE], None)


@pytest.mark.parametrize("kw", [dict(layer=-1), dict(layer=2), dict(table=None), dict(table=A + 2), dict(pps=0),
                                dict(pps=1 << 27), dict(n_seqs=-1), dict(lengths=None), dict(start=None),
                                dict(masks=None), dict(masks=A + 4), dict(n_rows=-1), dict(max_nodes=0),
                                dict(max_nodes=65), dict(heads=0), dict(heads=3), dict(q=None), dict(q=A + 2),
                                dict(ldq=255), dict(out=None), dict(ldo=255), dict(status=A + 1)])
def test_tree_attention_refuses(lib, kw):
    assert tree(lib, **kw) == q3tts.ERR_ARG


def test_tree_attention_limits(lib):
    assert tree(lib, heads=2 * 1025, ldq=1 << 20, ldo=1 << 20) == q3tts.ERR_UNSUPPORTED
    assert tree(lib, cache(n_pages=1 << 25)) == q3tts.ERR_UNSUPPORTED  # 2^32 rows


@pytest.mark.parametrize("kw", [dict(out=A), dict(out=A + 4), dict(out=A + 1024), dict(out=A + 8191 * 4),
                                dict(out=A + 1024, ldq=512), dict(q=A + 1024, out=A, ldo=512)])
def test_tree_attention_refuses_to_write_its_queries(lib, kw):
    a = dict(n_rows=40, out=A)
    a.update(kw)
    assert tree(lib, **a) == q3tts.ERR_ARG


@pytest.mark.parametrize("tile,us", [(-1, 100), (0, 0), (0, -5), (0, 2000001)])
def test_lose_tile_refuses(lib, tile, us):
    assert lib.q3tts_debug_lose_tile(tile, us) == q3tts.ERR_ARG


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_caches_are_checked(lib, bad, code):
    kv = cache(**bad)
    one = (C.c_int32 * 1)(0)
    two = (C.c_int32 * 1)(1)
    assert tree(lib, kv) == code
    assert lib.q3tts_copy_pages(C.byref(kv), one, two, 1, None) == code
    assert lib.q3tts_compact_rows(C.byref(kv), A, 4, 1, A, A, 4, A, None, None) == code


def test_no_work_is_no_error(lib):
    assert tree(lib, n_seqs=0) == q3tts.OK
    assert tree(lib, n_rows=0) == q3tts.OK
    assert lib.q3tts_copy_pages(C.byref(cache()), None, None, 0, None) == q3tts.OK
    assert lib.q3tts_compact_rows(C.byref(cache()), None, 4, 0, None, None, 4, None, None, None) == q3tts.OK
    assert lib.q3tts_reorder_rows(None, 0, None, None, 3, 2, 2, None, None) == q3tts.OK


@pytest.mark.parametrize("src,dst", [([0], [10]), ([10], [0]), ([-1], [0]), ([0], [-1]), ([0, 1], [2, 2]),
                                     ([0, 1], [1, 2]), ([3], [3])])
def test_copy_pages_refuses(lib, src, dst):
    s, d = (np.array(v, np.int32) for v in (src, dst))
    assert lib.q3tts_copy_pages(C.byref(cache()), s.ctypes.data, d.ctypes.data, len(src), None) == q3tts.ERR_ARG
    assert lib.q3tts_copy_pages(C.byref(cache()), None, d.ctypes.data, 1, None) == q3tts.ERR_ARG
    assert lib.q3tts_copy_pages(C.byref(cache()), s.ctypes.data, d.ctypes.data, -1, None) == q3tts.ERR_ARG


@pytest.mark.parametrize("args", [(None, 4, 1, A, A, 4, A), (A, 0, 1, A, A, 4, A), (A, 4, -1, A, A, 4, A),
                                  (A, 4, 1, None, A, 4, A), (A, 4, 1, A, None, 4, A), (A, 4, 1, A, A, -1, A),
                                  (A, 4, 1, A, A, 65, A), (A, 4, 1, A, A, 4, None), (A, 4, 1, A, A, 4, A + 1)])
def test_compact_rows_refuses(lib, args):
    assert lib.q3tts_compact_rows(C.byref(cache()), *args, None, None) == q3tts.ERR_ARG


BEAM = ["logits", "ld", "ids", "groups", "beams", "vocab", "scores", "finished", "history", "eos", "special",
        "penalty", "k", "tokens", "parents", "out", "ws", "ws_bytes"]


def beam(lib, **kw):
    a = dict(logits=A, ld=100, ids=None, groups=2, beams=4, vocab=100, scores=A + 4096, finished=None, history=None,
             eos=-1, special=0, penalty=1.0, k=4, tokens=A + 8192, parents=A + 12288, out=A + 16384, ws=A + 20480, ws_bytes=1 << 30)
    a.update(kw)
    return lib.q3tts_beam_select(*[a[n] for n in BEAM], None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), q3tts.ERR_ARG), (dict(logits=A + 2), q3tts.ERR_ARG), (dict(ld=99), q3tts.ERR_ARG),
    (dict(groups=-1), q3tts.ERR_ARG), (dict(beams=0), q3tts.ERR_ARG), (dict(vocab=0), q3tts.ERR_ARG),
    (dict(k=0), q3tts.ERR_ARG), (dict(scores=None), q3tts.ERR_ARG), (dict(tokens=None), q3tts.ERR_ARG),
    (dict(parents=None), q3tts.ERR_ARG), (dict(out=None), q3tts.ERR_ARG), (dict(eos=100), q3tts.ERR_ARG),
    (dict(special=101), q3tts.ERR_ARG), (dict(penalty=0.0), q3tts.ERR_ARG), (dict(finished=A), q3tts.ERR_ARG),
    (dict(ws=A + 4), q3tts.ERR_ARG),
    (dict(out=A + 4096 + 4), q3tts.ERR_ARG), (dict(out=A + 4096, k=3), q3tts.ERR_ARG),
    (dict(beams=33), q3tts.ERR_UNSUPPORTED), (dict(k=33), q3tts.ERR_UNSUPPORTED),
    (dict(vocab=(1 << 24) + 1, ld=1 << 25), q3tts.ERR_UNSUPPORTED)])
def test_beam_select_refuses(lib, kw, code):
    assert beam(lib, **kw) == code


@pytest.mark.parametrize("row,kw,code", [
    ((None, A, 8, 8, 8), {}, q3tts.ERR_ARG), ((A, None, 8, 8, 8), {}, q3tts.ERR_ARG),
    ((A, A + 1024, 8, 7, 8), {}, q3tts.ERR_ARG), ((A, A + 1024, 8, 8, 4), {}, q3tts.ERR_ARG),
    ((A, A + 8, 8, 8, 8), {}, q3tts.ERR_ARG),               # overlaps, not in place
    ((A, A, 8, 8, 16), {}, q3tts.ERR_ARG),                  # in place with another stride
    ((A, A, 8, 8, 8), dict(b_in=3), q3tts.ERR_ARG),         # in place with other beams
    ((A, A + 1024, 8, 8, 8), dict(parents=None), q3tts.ERR_ARG),
    ((A, A + 1024, 8, 8, 8), dict(ids=A, b_in=3), q3tts.ERR_ARG),
    ((A, A + 1024, 8, 8, 8), dict(b_in=0), q3tts.ERR_ARG),
    ((A, A + 1024, 8, 8, 8), dict(b_in=33), q3tts.ERR_UNSUPPORTED),
    ((A, A + 1024, 8, 8, 8), dict(groups=2048), q3tts.ERR_UNSUPPORTED)])
def test_reorder_rows_refuses(lib, row, kw, code):
    a = dict(ids=None, parents=A, groups=2, b_in=4, b_out=4)
    a.update(kw)
    s = q3tts.Rows(*row)
    assert lib.q3tts_reorder_rows(C.byref(s), 1, a["ids"], a["parents"], a["groups"], a["b_in"], a["b_out"], None,
                                  None) == code


def test_handle_calls_refuse_null(lib):
    ids = (C.c_int32 * 2)(1, 2)
    sp = q3tts.Sampling()
    assert lib.q3tts_fork(None, 0, ids, 2) == q3tts.ERR_ARG
    assert lib.q3tts_tree_step(None, 0, A, ids, 1, None, None) == q3tts.ERR_ARG
    assert lib.q3tts_tree_accept(None, 0, ids, 1) == q3tts.ERR_ARG
    assert lib.q3tts_beam_frame(None, C.byref(sp), ids, 1, 2, A, A, A, None) == q3tts.ERR_ARG


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    pool = torch.zeros((1, 2, 2, 1, 16, 64))
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(q3tts.Q3TTSError):
        q3tts.copy_pages(pool, [0], [1])
    with pytest.raises(q3tts.Q3TTSError):
        q3tts.compact_rows(pool, i[None], i, i[None], i)
    with pytest.raises(q3tts.Q3TTSError):
        q3tts.tree_attention(pool, 0, i[None], i, torch.zeros(2, dtype=torch.int32), i.long(), torch.zeros(1, 1, 64))
    with pytest.raises(q3tts.Q3TTSError):
        q3tts.beam_select(torch.zeros(1, 1, 8), torch.zeros(1, 1))
    with pytest.raises(q3tts.Q3TTSError):
        q3tts.reorder_rows([torch.zeros(1, 1, 8)], [torch.zeros(1, 1, 8)], i[None])


def reorder(lib, rows, groups=2, b_in=2, b_out=2, ids=None, parents=A + (1 << 30)):
    sets = (q3tts.Rows * len(rows))(*[q3tts.Rows(*r) for r in rows])
    return lib.q3tts_reorder_rows(sets, len(rows), ids, parents, groups, b_in, b_out, None, None)


X, Y = A, A + 4096


@pytest.mark.parametrize("rows", [
    [(X, Y, 64, 64, 64), (Y, X, 64, 64, 64)],                  # two buffers exchanged
    [(X, X, 64, 64, 64), (X, X, 64, 64, 64)],                  # one buffer twice, in place
    [(X, Y, 64, 64, 64), (X + 8192, Y + 64, 64, 64, 64)],      # one dst, a row on
    [(X, X, 64, 64, 64), (X + 100, Y, 64, 64, 64)],            # a dst that another set reads
    [(X, Y, 64, 64, 64), (Y + 250, Y + 4096, 8, 8, 8)],        # by its last bytes
    [(X, X, 16, 64, 64), (X + 8, X + 8, 16, 64, 64)],          # fields of a record that overlap
    [(X, X, 16, 64, 64), (X + 16, Y, 16, 40, 40)],             # other strides: rows meet at the second
    [(X, Y, 64, 64, 64)] + [(X + 8192 + 4096 * i, Y + 4096 * i, 0, 0, 0) for i in range(8)] + [(Y, X + 65536, 4, 4, 4)]])
def test_reorder_rows_refuses_sets_that_meet(lib, rows):
    """All sets of a call may run at once, so one may not write what another reads or writes."""
    assert reorder(lib, rows) == q3tts.ERR_ARG
    assert reorder(lib, rows[::-1]) == q3tts.ERR_ARG


def test_reorder_rows_refuses_by_ids_and_parents(lib):
    """Rows by ids: the same rows of equally spaced buffers.  A dst on the parents."""
    for rows in ([(X, Y, 64, 64, 64), (Y, X, 64, 64, 64)], [(X, X, 64, 64, 64)] * 2, [(X, X + 32, 64, 64, 64)]):
        assert reorder(lib, rows, ids=A) == q3tts.ERR_ARG
    assert reorder(lib, [(X, Y, 4, 4, 4)], parents=Y) == q3tts.ERR_ARG
    assert reorder(lib, [(X, Y, 4, 4, 4)], parents=Y + 12) == q3tts.ERR_ARG


def test_reorder_rows_tells_rows_that_meet_from_rows_between_rows(lib):
    """Against the bytes themselves, for random sets.  (What is not refused ends at the
    launch: there is no GPU here.  With one the addresses would be followed.)"""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    rng = np.random.default_rng(2)
    seen = set()
    for _ in range(3000):
        groups, b_in, b_out = (int(rng.integers(1, 4)) for _ in range(3))
        many = int(rng.integers(1, 3)) if rng.random() < 0.8 else 10
        rows, bad, marks = [], False, {}
        for i in range(many):
            nb = int(rng.integers(1, 7))
            st = int(rng.choice([nb, 8, 12, 24]))
            st = max(st, nb)
            span = 60 if many < 9 else 900
            src = A + int(rng.integers(0, span))
            if b_in == b_out and rng.random() < 0.4:
                row = (src, src, nb, st, st)
            else:
                row = (src, A + int(rng.integers(0, span)), nb, st, max(nb, int(rng.choice([st, 12]))))
                if row[1] == src:
                    continue
            rows.append(row)
            read = {src + r * row[3] + e for r in range(groups * b_in) for e in range(nb)}
            write = {row[1] + r * row[4] + e for r in range(groups * b_out) for e in range(nb)}
            bad = bad or (row[0] != row[1] and bool(read & write))
            for o_read, o_write in marks.values():
                bad = bad or bool(write & o_read) or bool(write & o_write) or bool(read & o_write)
            marks[i] = read, write
        if not rows:
            continue
        rc = reorder(lib, rows, groups, b_in, b_out)
        assert rc == (q3tts.ERR_ARG if bad else q3tts.ERR_CUDA), rows
        seen.add((bad, len(rows) > 8))
    assert len(seen) == 4
