"""NaN in the cache reaches every row that attends it, also where the row's
tokens are joined from parts: softmax over a NaN score is NaN everywhere."""
import pytest
import torch

from ._ops import BS, ok
from .test_gpu_shared import Shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (12, 2), (2, 2)])
@pytest.mark.parametrize("own", [1, 20, 40, 500, 6000])
def test_key_of_an_own_token_behind_a_prefix(pa, own, Hq, Hkv, out_dtype):
    """(One tile, a whole segment of the own-token decode, and a cut one.)"""
    c = Shared(pa, [(12, [20, own, 3])], [30], Hq, Hkv, torch.bfloat16, seed=21, order="given")
    i, t, G = 1, 12 * BS + own - 1, Hq // Hkv
    clean = c.call(out_dtype)
    c.pool.k[int(c.tables[i, t // BS]), 1, t % BS, 5] = float("nan")
    out = c.call(out_dtype)
    assert torch.isnan(out[i, G:]).all()
    out[i, G:] = clean[i, G:]
    assert torch.equal(out, clean)
    ok(pa, c.pool)
    c.pool.close()
