"""The 8-bit cache's write and read in calls of many sequences that leave the most rows of a
sequence to its default."""
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


@pytest.mark.parametrize("seqs,rows,kvh,block", [(1024, 16, 4, 1), (4096, 64, 1, 16)])
def test_many_sequences_without_a_bound_on_their_rows(q3, seqs, rows, kvh, block):
    """2^27 warps and more, nearly all of them without rows: as with the bound given."""
    import torch
    rng = np.random.default_rng(51)
    n, page = seqs * rows, 16
    pages = seqs * (rows // page)
    table = torch.from_numpy(rng.permutation(pages).astype(np.int32).reshape(seqs, -1)).cuda()
    lens, start = ku.ints([0] * seqs), ku.ints(np.arange(seqs + 1) * rows)
    k, v = (t8.randn(rng, (n, kvh, 64), torch.bfloat16) for _ in range(2))
    got = []
    for most in (rows, None):
        pool = torch.zeros((1, pages, 2, kvh, page, 64), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        scales = torch.zeros((1, pages, 2, kvh, page // block), dtype=torch.uint8, device="cuda")
        out = tuple(torch.zeros_like(k) for _ in range(2))
        q3.kv8_write(pool, scales, 0, table, lens, start, k, v, max_rows=most)
        q3.kv8_read(pool, scales, 0, table, lens, start, max_rows=most, out=out)
        got.append((pool.view(torch.uint8), scales, *out))
    assert bool((got[0][1] != 0).all()) and all(torch.equal(a, b) for a, b in zip(*got))
