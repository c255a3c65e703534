"""The 8-bit cache's attention over queries that are not finite or very large or small,
in both of its kernels."""
import math

import numpy as np
import pytest

from tests import test_gpu_kv8 as t8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from autoregressive_tts_decode_gb300 import build, q3tts
    build.build()
    return q3tts


@pytest.mark.parametrize("rows,heads,kvh,length,seqs", t8.SHAPES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("tree", [True, False])
def test_a_query_that_is_not_finite(q3, rows, heads, kvh, length, seqs, dtype, tree):
    """NaN, +infinity or -infinity in one element of a head's query: that head's output of that row is
    NaN, the others are within their bound (rows of a tile follow their largest scores together, so that the others'
    roundings may change).  Codes of one sign beside it, so that a product with an infinity has one sign at every
    position."""
    import torch
    c = t8.attend_case(np.random.default_rng(31), [length] * seqs, [rows] * seqs, heads, kvh, 128, 16, 16, dtype, tree)
    c["codes"][..., 5] = np.where(c["codes"][..., 5] & 127 == t8.ku.NAN, t8.ku.NAN, c["codes"][..., 5] & 0x3F | 8)
    want, tol = t8.ku.attention_reference(c["codes"], c["powers"], 1, c["table"], c["lens"], c["rows"], c["masks"], c["q"])
    n = rows * seqs
    for i, bad in enumerate((math.nan, math.inf, -math.inf)):
        row, head = (n // 2 + i) % n, i % heads
        q = c["q"].clone()
        q[row, head, 5] = bad
        out = t8.run_attention(q3, dict(c, q=q))
        same = torch.ones((n, heads), dtype=torch.bool, device="cuda")
        same[row, head] = False
        assert bool(torch.isnan(out[row, head]).all()), bad
        assert bool(((out.double() - want).abs() <= tol)[same].all())


@pytest.mark.parametrize("seqs", [1, 60])
@pytest.mark.parametrize("rows", [1, 7, 64])
def test_a_query_that_is_not_finite_and_sees_nothing(q3, rows, seqs):
    """Zeroes, as of any row that sees nothing."""
    import torch
    c = t8.attend_case(np.random.default_rng(32), [0] * seqs, [rows] * seqs, 4, 2, 64, 16, 8, "float32", True)
    c["masks"] = [0 if i % rows == rows - 1 else m for i, m in enumerate(c["masks"])]
    want = t8.run_attention(q3, c)
    c["q"][rows - 1::rows, 0, 0] = math.nan
    c["q"][rows - 1::rows, 1] = math.inf
    out = t8.run_attention(q3, c)
    assert torch.equal(out, want) and bool((out[rows - 1::rows] == 0).all())


@pytest.mark.parametrize("rows,heads,kvh,length,seqs", t8.SHAPES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("size,byte", [(126, 1), (120, 7), (-100, 227), (-120, 247), (-127, 254)])
def test_queries_at_either_end_of_the_range(q3, rows, heads, kvh, length, seqs, dtype, size, byte):
    """Queries of up to 2^128 and down into the subnormals, over keys whose powers make the
    scores ordinary ones."""
    import torch
    c = t8.attend_case(np.random.default_rng(33), [length] * seqs, [rows] * seqs, heads, kvh, 128, 16, 16, dtype, False)
    codes, powers = c["codes"][:, :, 0], c["powers"][:, :, 0]
    c["codes"][:, :, 0] = np.where(codes & 127 == t8.ku.NAN, t8.ku.NAN, codes & 0xBF)  # below 2 in size
    c["powers"][:, :, 0] = np.where(powers == 255, 255, byte)
    q = t8.randn(np.random.default_rng(34), c["q"].shape, torch.float64).clamp(-3.9, 3.9) * 2.0 ** size
    c["q"] = q.to(t8.dt(dtype))
    assert bool(c["q"].isfinite().all()) and (size < 126 or float(c["q"].abs().max()) >= 2.0 ** 127)
    t8.check_attention(c, t8.run_attention(q3, c))
