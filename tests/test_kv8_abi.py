"""Refusals of the 8-bit cache's entries without a GPU: every argument check answers
before any device work (the pointers are made up and never followed)."""
import ctypes as C
import os
import re

import pytest

from autoregressive_tts_decode_gb300 import build, q3tts

A = 1 << 40  # a made-up device address


@pytest.fixture(scope="module")
def lib():
    build.build()
    return q3tts.load()


def header():
    return open(os.path.join(os.path.dirname(build.HERE), "include", "q3tts_kv8.h")).read()


def cache(**kw):
    f = dict(codes=A, powers=A + (1 << 30) + 1, layers=2, n_pages=10, n_kv_heads=2, page_size=16, head_dim=64, block=8)
    f.update(kw)
    return C.byref(q3tts.KV8Cache(*[f[n] for n, _ in q3tts.KV8Cache._fields_]))


ROWS = dict(table=A, lengths=A, start=A, status=None, layer=0, pps=4, n_seqs=2, dtype=q3tts.F32, n_rows=8, max_rows=4)
PAIR = dict(a=A, lda=256, b=A + 65536, ldb=256)


def call(fn, kv, before, pair, after, kw):
    rows, args = dict(ROWS), {**before, **pair, **after, "stream": None}
    assert set(kw) <= set(rows) | set(args)
    rows.update((n, v) for n, v in kw.items() if n in rows)
    args.update((n, v) for n, v in kw.items() if n in args)
    return fn(kv, C.byref(q3tts.KV8Rows(*rows.values())), *args.values())


def write(lib, kv=None, **kw):
    return call(lib.q3tts_kv8_write, cache() if kv is None else kv, {}, PAIR, {}, kw)


def read(lib, kv=None, **kw):
    return call(lib.q3tts_kv8_read, cache() if kv is None else kv, dict(path=None), PAIR, {}, kw)


def attend(lib, kv=None, **kw):
    return call(lib.q3tts_kv8_attention, cache() if kv is None else kv, dict(masks=None), PAIR, dict(heads=4), kw)


CALLS = [write, read, attend]


def test_exports_every_declared_function(lib):
    names = set(re.findall(r"^(?:int|size_t) (q3tts_[a-z0-9_]+)\(", header(), re.M))
    assert names == set(q3tts.KV8_EXPORTS) and not names & (set(q3tts.EXPORTS) | set(q3tts.BRANCH_EXPORTS))
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("name,struct,packed", [("q3tts_kv8_cache", q3tts.KV8Cache, q3tts._CACHE8),
                                                ("q3tts_kv8_rows", q3tts.KV8Rows, q3tts._ROWS8)])
def test_struct_layouts_match_header(name, struct, packed):
    body = re.search(r"typedef struct " + name + r" \{(.*?)\} " + name, header(), re.S).group(1)
    names = [n.strip().split()[-1].lstrip("*") for d in body.split(";") if d.strip() for n in d.split(",")]
    assert names == [f[0] for f in struct._fields_]
    assert packed.size == C.sizeof(struct)


@pytest.mark.parametrize("fn", CALLS)
@pytest.mark.parametrize("bad,code", [
    (dict(codes=None), q3tts.ERR_ARG), (dict(codes=A + 8), q3tts.ERR_ARG), (dict(powers=None), q3tts.ERR_ARG),
    (dict(layers=0), q3tts.ERR_ARG), (dict(n_pages=0), q3tts.ERR_ARG), (dict(n_kv_heads=0), q3tts.ERR_ARG),
    (dict(page_size=0), q3tts.ERR_ARG), (dict(block=0), q3tts.ERR_ARG), (dict(block=5), q3tts.ERR_ARG),
    (dict(block=32), q3tts.ERR_ARG), (dict(head_dim=96), q3tts.ERR_UNSUPPORTED)])
def test_caches_are_checked(lib, fn, bad, code):
    assert fn(lib, cache(**bad)) == code
    assert fn(lib, C.POINTER(q3tts.KV8Cache)()) == q3tts.ERR_ARG


def test_no_rows_at_all(lib):
    assert lib.q3tts_kv8_write(cache(), None, A, 256, A, 256, None) == q3tts.ERR_ARG
    assert lib.q3tts_kv8_read(cache(), None, None, A, 256, A, 256, None) == q3tts.ERR_ARG
    assert lib.q3tts_kv8_attention(cache(), None, None, A, 256, A, 256, 4, None) == q3tts.ERR_ARG


@pytest.mark.parametrize("fn", CALLS)
@pytest.mark.parametrize("kw", [
    dict(layer=-1), dict(layer=2), dict(table=None), dict(table=A + 2), dict(pps=0), dict(pps=1 << 27), dict(n_seqs=-1),
    dict(lengths=None), dict(lengths=A + 1), dict(start=None), dict(start=A + 2), dict(n_rows=-1), dict(max_rows=0),
    dict(dtype=q3tts.FP8), dict(dtype=-1), dict(status=A + 1), dict(a=None), dict(a=A + 2), dict(b=None), dict(b=A + 65538),
    dict(lda=127), dict(ldb=127), dict(a=A + 1, dtype=q3tts.BF16), dict(b=A + 65537, dtype=q3tts.BF16)])
def test_calls_refuse(lib, fn, kw):
    assert fn(lib, **kw) == q3tts.ERR_ARG


@pytest.mark.parametrize("fn", CALLS)
def test_no_work_is_no_error(lib, fn):
    assert fn(lib, n_seqs=0, table=None, a=None) == q3tts.OK
    assert fn(lib, n_rows=0, lengths=None, b=None) == q3tts.OK


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), q3tts.ERR_ARG), (dict(heads=3), q3tts.ERR_ARG), (dict(masks=A + 4), q3tts.ERR_ARG),
    (dict(masks=A, max_rows=65), q3tts.ERR_ARG), (dict(lda=255), q3tts.ERR_ARG), (dict(ldb=255), q3tts.ERR_ARG),
    (dict(heads=2 * 1025, lda=1 << 20, ldb=1 << 20, b=A + (1 << 30)), q3tts.ERR_UNSUPPORTED)])
def test_attention_refuses(lib, kw, code):
    assert attend(lib, **kw) == code


def test_attention_counts_the_caches_rows(lib):
    assert attend(lib, cache(n_pages=1 << 25)) == q3tts.ERR_UNSUPPORTED  # 2^32 rows


@pytest.mark.parametrize("kw", [dict(b=A), dict(b=A + 4), dict(b=A + 1024), dict(b=A + 1024, lda=512),
                                dict(a=A + 1024, b=A, ldb=512), dict(b=A + 2, dtype=q3tts.BF16)])
def test_attention_refuses_to_write_its_queries(lib, kw):
    assert attend(lib, n_rows=40, **kw) == q3tts.ERR_ARG


@pytest.mark.parametrize("kw", [dict(b=A), dict(b=A + 256), dict(b=A + 1024), dict(b=A + 510, dtype=q3tts.BF16)])
def test_read_refuses_keys_over_values(lib, kw):
    assert read(lib, n_rows=40, **kw) == q3tts.ERR_ARG
    assert read(lib, path=A + 2) == q3tts.ERR_ARG
