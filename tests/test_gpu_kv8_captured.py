"""A step over the 8-bit cache as a captured graph: what each replay writes, attends and reads
is the definition's on the cache as it was before that replay."""
import numpy as np
import pytest

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


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("lens,rows,heads,kvh,hd,block", [([130, 700], [1, 1], 16, 8, 128, 16), ([15, 0, 333], [1, 1, 1], 4, 2, 64, 8),
                                                          ([200, 40], [70, 90], 4, 2, 128, 16), ([31] * 90, [1] * 90, 4, 2, 64, 16)])
def test_replays_write_what_they_are_given(q3, dtype, lens, rows, heads, kvh, hd, block):
    """Write, attention and read in one graph on a side stream, replayed on new rows whose sizes rise and
    fall (codes held in a block are rounded again), at lengths that go on by the rows written.
    The write's codes and powers are compared with its definition on a copy taken before the replay."""
    import torch
    rng, t, page, steps = np.random.default_rng(61), t8.dt(dtype), 16, 4
    codes, powers, table = ku.cache(rng, [a + steps * b for a, b in zip(lens, rows)], page, block, 2, kvh, hd, 118, 122)
    pool, scales, tab = ku.to_gpu(codes, powers, table)
    n, most = sum(rows), max(rows)
    now = list(lens)
    ln, start = ku.ints(now), ku.ints(ku.starts(rows))
    k, v, q = (torch.zeros((n, h, hd), dtype=t, device="cuda") for h in (kvh, kvh, heads))
    out, back = torch.empty_like(q), (torch.empty_like(k), torch.empty_like(v))

    def calls():
        q3.kv8_write(pool, scales, 1, tab, ln, start, k, v, max_rows=most)
        q3.kv8_attention(pool, scales, 1, tab, ln, start, q, max_rows=most, out=out)
        q3.kv8_read(pool, scales, 1, tab, ln, start, max_rows=most, out=back)

    warm = pool.view(torch.uint8).clone(), scales.view(torch.uint8).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()  # (so that nothing is looked up for the first time in the capture)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls()
    pool.view(torch.uint8).copy_(warm[0])
    scales.view(torch.uint8).copy_(warm[1])
    for step in range(steps):
        ln.copy_(ku.ints(now))
        for x, size in ((k, 2.0 ** (3 * step % 7)), (v, 2.0 ** (5 * step % 7)), (q, 2.0 ** -3)):
            x.copy_(t8.randn(rng, x.shape, torch.float32) * size)
        before = pool.view(torch.uint8).cpu().numpy().copy(), scales.view(torch.uint8).cpu().numpy().copy()
        out.fill_(-7.5)
        graph.replay()
        torch.cuda.synchronize()
        want, wpow = ku.write_reference(*before, 1, table, now, rows, k.double().cpu().numpy(), v.double().cpu().numpy())
        after, apow = pool.view(torch.uint8).cpu().numpy(), scales.view(torch.uint8).cpu().numpy()
        assert np.array_equal(apow, wpow) and t8.same_values(pool, want)
        assert not np.array_equal(after, before[0])
        ref, tol = ku.attention_reference(after, apow, 1, table, now, rows, None, q)
        assert bool(((out.double() - ref).abs() <= tol).all())
        at = 0
        for s, m in enumerate(rows):
            c, p = ku.values(after, apow, 1, table, s, now[s] + np.arange(m))
            for j in (0, 1):
                assert torch.equal(back[j][at:at + m], torch.from_numpy(c[j] * p[j][..., None]).cuda().float().to(t))
            at += m
        now = [a + b for a, b in zip(now, rows)]
