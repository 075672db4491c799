"""Both sides of the launch rules of the 8-bit decode: the rule chooses the plan, not the result."""
import numpy as np
import pytest

from ._ops import BS
from ._ops8 import ok8
from .test_gpu_decode8 import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


@pytest.mark.parametrize("Hq,Hkv,B", [(24, 3, 21), (16, 4, 16), (8, 8, 9), (38, 38, 4), (24, 3, 51)])
@pytest.mark.parametrize("width", [47, 48, 49])
def test_tables_at_the_limit_of_many_segments(pa, Hq, Hkv, B, width):
    """63, 64, 72, 152 and 153 segments, tables of 48 blocks and one less and more, ragged and alike."""
    rng = np.random.default_rng(width + B)
    for alike in (True, False):
        lens = np.full(B, width * BS) if alike else rng.integers(0, width * BS + 1, B)
        c = Case(pa, lens.tolist(), Hq, Hkv, "int8" if alike else "e4m3", seed=B, width=width)
        c.check(c.call())
        ok8(pa, c.pool)
