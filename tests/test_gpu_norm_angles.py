"""The rotation inside the norm appends keeps 32 bits.

Rows of ones in the first halves and zeros in the second leave the cosine and the sine of each angle as outputs.  For
positions below 2^12 the angle in turns is one rounding (2^-26 turns, 2^-23.3 rad) and a remainder below 2^-36 off; the
cosine and the sine of it one unit (2^-24) at most: 2^-22.5 together, beside half a step of fp16 (2^-25 at the least)."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, half_step, to64
from ._ops8 import type8
from .test_gpu_norm_rope import Tokens, weight

pytestmark = pytest.mark.gpu
DT = torch.float16


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


def unit_rows(rng, n, Hq, Hkv):
    t = Tokens(rng, n, Hq, Hkv, DT, 128, 1, False)
    t.pos = rng.integers(0, 1 << 12, (1, n)).astype(np.int32)
    for x in (t.q, t.k):
        x[:, :, :64], x[:, :, 64:] = 1.0, 0.0
    return t


def check(got, t):
    a = t.pos[0].astype(np.float64)[:, None] * t.inv.astype(np.float64)
    want = np.concatenate([np.cos(a), np.sin(a)], 1)[:, None]
    bad = np.abs(got - want) > half_step(DT) * np.abs(want) + 2.0 ** -25 + 2.0 ** -22.5
    assert not bad.any(), (int(bad.sum()), float(np.log2(np.abs(got - want)[bad].max())))


@pytest.mark.parametrize("n", [40, 3000])
def test_rows_without_a_weight_beside_normed_ones(pa, n):
    rng = np.random.default_rng(n)
    pool = pa.Pool(-(-n // BS), 8, DT)
    for norms in "qk":
        t = unit_rows(rng, n, 32, 8)
        w = weight(rng, DT)
        pa.pa_norm_rope_append(pool, *t.args(w if norms == "q" else None, w if norms == "k" else None, np.arange(n)))
        rows = to64(pool.k).transpose(0, 2, 1, 3).reshape(-1, 8, D)[:n]
        check(rows if norms == "q" else to64(t.q_out), t)
    pool.close()


@pytest.mark.parametrize("n", [40, 3000])
def test_query_rows_next_to_the_8_bit_cache(pa, n):
    rng = np.random.default_rng(n + 1)
    pool = pa.Pool8(-(-n // BS), 8, type8("e4m3"))
    w = weight(rng, DT)
    for wk in (w, None):
        t = unit_rows(rng, n, 32, 8)
        pa.pa_norm_rope_append8(pool, *t.args(None, wk, np.arange(n)))
        check(to64(t.q_out), t)
    pool.close()
