"""Host side of the 8-bit cache: sizes that are refused, and what the header says of its roundings, on the tests' own
64-bit definitions."""
import ctypes

import numpy as np
import pytest

import paged_kv_cache_227_gb300 as pa

from ._ops8 import KINDS, decode8, write8


def test_pools_whose_blocks_pass_32_bits_are_refused():
    """Offsets inside a block are 32-bit: 2^19 heads are a block of 2^31 bytes."""
    h = ctypes.c_void_p()
    for create, dtype in ((pa.lib.pa_pool_create, pa.PA_BF16), (pa.lib.pa_pool8_create, pa.PA_INT8)):
        for heads in (1 << 19, (1 << 24) + 3, (1 << 27) - 1):
            assert create(1, 16, heads, 128, dtype, ctypes.byref(h)) == pa.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kind", KINDS)
def test_bounds_that_the_header_states(kind):
    """Written afresh: int8 half a scale, at most 1/127 of the largest magnitude (2^-7 is less: reached just above a
    power of two of 63.5); e4m3 2^-4 of a value or 2^-10 of the scale.  Written row by row, from small to large, every
    rounding together: below a scale; below 2^-4 of a value + 2^-9 of the scale."""
    rng = np.random.default_rng(7)
    afresh = over = most = 0.0
    for trial in range(200):
        rows = rng.uniform(-1, 1, (16, 1, 128)) * 2.0 ** np.sort(rng.uniform(-9, 5, 16))[:, None, None]
        if trial % 2:  # every row just above what the scale before holds
            rows *= 63.5 * 1.001 * 2.0 ** (np.arange(16) // 2)[:, None, None] / np.abs(rows).max((1, 2), keepdims=True)
        empty = np.zeros((1, 1, 16, 128), np.uint8), np.zeros((1, 1), np.uint8)
        codes, exps = write8(*empty, rows, np.arange(16), kind)
        scale, top = 2.0 ** (float(exps[0, 0]) - 127), np.abs(rows).max()
        err = np.abs(decode8(codes[0, 0], kind) * scale - rows[:, 0])
        if kind == "int8":
            assert err.max() <= scale / 2 and err.max() <= top / 127
            afresh = max(afresh, err.max() / top)
        else:
            assert (err <= np.maximum(2.0 ** -4 * np.abs(rows[:, 0]), 2.0 ** -10 * scale)).all()
        codes, exps = empty
        for r in range(16):
            before = int(exps[0, 0])
            codes, exps = write8(codes, exps, rows[r:r + 1], np.array([r]), kind)
            assert r == 0 or exps[0, 0] >= before
        scale = 2.0 ** (float(exps[0, 0]) - 127)
        err = np.abs(decode8(codes[0, 0], kind) * scale - rows[:, 0])
        bound = scale if kind == "int8" else 2.0 ** -4 * np.abs(rows[:, 0]) + 2.0 ** -9 * scale
        assert (err < bound).all()
        most = max(most, (err / scale).max())
    if kind == "int8":
        assert afresh > 2.0 ** -7 and most > 0.5, "neither 2^-7 of the largest magnitude nor half a scale would hold"
