"""The 8-bit cache's attention where scores and powers of two of the values are far apart in
one sequence: the softmax's sum counts every position, whatever its value's power."""
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


def by_first_element(rng, rows, heads, kvh, length, seqs, dtype, scale):
    """A case whose scores, in units of log2, are scale x the first code of a key (power 1, the
    others zero)."""
    import torch
    c = t8.attend_case(rng, [length] * seqs, [rows] * seqs, heads, kvh, 128, 16, 16, dtype, False)
    c["codes"][:, :, 0] = 0
    c["powers"][:, :, 0] = np.where(c["powers"][:, :, 0] == 255, 255, 127)
    c["powers"][:, :, 1] = np.where(c["powers"][:, :, 1] == 255, 255, 127)
    c["q"] = torch.zeros_like(c["q"])
    c["q"][:, :, 0] = scale * math.sqrt(128) / math.log2(math.e)
    return c


def code_of(value):
    return int(np.flatnonzero(t8.ku.VALUES == value)[0])


@pytest.mark.parametrize("rows,heads,kvh,tiles,seqs", [(1, 4, 2, 6, 1), (1, 4, 2, 48, 1), (1, 16, 8, 6, 90), (4, 8, 2, 12, 70), (64, 4, 2, 12, 3),
                                                       (64, 4, 2, 6, 60)])
def test_scores_of_zero_values(q3, rows, heads, kvh, tiles, seqs):
    """Blocks of nothing but zeroes (power byte 0) whose scores are 127.5 above the ordinary ones
    before them and 16 below those that follow: sums of weights relative to the ordinary ones would pass fp32's range."""
    rng = np.random.default_rng(41)
    c = by_first_element(rng, rows, heads, kvh, 128 * tiles, seqs, "float32", 127.5 / 128)
    for s in range(seqs):
        for j in range(8 * tiles):  # pages of 16, one block each
            pg, kind = c["table"][s, j], j // 8 % 6
            if 0 < kind < 5:
                c["codes"][:, pg, 0, :, :, 0] = code_of(128.0)
                c["codes"][:, pg, 1], c["powers"][:, pg, 1] = 0, 0
            elif kind == 5:
                c["codes"][:, pg, 0, :, :, 0] = code_of(144.0)
    t8.check_attention(c, t8.run_attention(q3, c))


@pytest.mark.parametrize("rows,heads,kvh,length,seqs,gap", [(1, 2, 1, 60000, 1, 28), (4, 2, 1, 60000, 1, 28), (1, 8, 8, 20000, 20, 26),
                                                            (64, 2, 1, 60000, 1, 28), (64, 4, 2, 20000, 20, 26)])
def test_zero_values_beside_large_ones(q3, rows, heads, kvh, length, seqs, gap):
    """One position's value of power 2^40 among zeroes (power byte 0) whose scores are `gap` lower: each of
    these has a weight of 2^-gap in the sum.  The bound: the large value's weight is in its product and in the sum alike,
    so what is left are the exponential's error (2^-21 of it), fp32 roundings (2^-24 each, a few) and the
    fixed-point steps (2^-27): 2^-19 together; and the sum's own roundings: the thread that has the large weight adds one
    for each tile of 128 positions, each sum half a step (2^-24) off at most (all of a weight of 2^-26, as of 154 tiles
    of the third case, 2.3e-6).  Without the zeroes' weights the result is 2^-12 off."""
    c = by_first_element(np.random.default_rng(42), rows, heads, kvh, length, seqs, "float32", 1.0)
    c["codes"][:, :, 1] = np.where(c["codes"][:, :, 1] & 127 == t8.ku.NAN, t8.ku.NAN, 0)
    c["powers"][:, :, 1] = np.where(c["powers"][:, :, 1] == 255, 255, 0)
    for s in range(seqs):
        pos = length * (s + 1) // (seqs + 2)
        pg, slot = c["table"][s, pos // 16], pos % 16
        c["codes"][:, pg, 0, :, slot, 0] = code_of(float(gap))
        c["codes"][:, pg, 1, :, slot] = np.random.default_rng(s).integers(64, 120, c["codes"].shape[-1])
        c["powers"][:, pg, 1] = 167
    out = t8.run_attention(q3, c).double()
    want, _ = t8.ku.attention_reference(c["codes"], c["powers"], 1, c["table"], c["lens"], c["rows"], None, c["q"])
    assert bool(((out - want).abs() <= (2.0 ** -19 + -(-length // 128) * 2.0 ** -24) * want.abs()).all()), float(((out - want) / want).abs().max())
