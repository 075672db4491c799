"""NaN in the cache reaches every row that attends it, also where the row's
tokens are joined from parts: softmax over a NaN score is NaN everywhere, and a
weight of zero times a NaN value is NaN."""
import pytest
import torch

from ._ops import BS, cuda, ok
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


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (12, 2)])
@pytest.mark.parametrize("where", ["prefix", "own", "own, cut"])
def test_value_of_a_token_whose_weight_underflows(pa, where, Hq, Hkv):
    """One token of the other part takes all the weight (256 above everything
    else): the part with the NaN value has weight 2^-300, which is 0 in 32 bits,
    and 0 * NaN is NaN, as in the plain decode."""
    own = 3000 if where == "own, cut" else 40
    c = Shared(pa, [(12, [20, own])], [], Hq, Hkv, torch.bfloat16, seed=22, order="given")
    i, G = 1, Hq // Hkv
    c.q[i, :G] = 1.0
    heavy, bad = (12 * BS + own - 1, 2 * BS + 5) if where == "prefix" else (3 * BS, 12 * BS + 7)
    c.pool.k[int(c.tables[i, heavy // BS]), 0, heavy % BS] = 4.0
    clean = c.call(scale=0.5)
    assert torch.isfinite(clean).all()
    c.pool.v[int(c.tables[i, bad // BS]), 0, bad % BS, 7] = float("nan")
    out = c.call(scale=0.5)
    plain = torch.empty_like(out)
    pa.pa_decode_split(c.pool, c.q, cuda(c.tables), cuda(c.lens), 0.5, plain)
    assert torch.isnan(plain[i, :G, 7]).all()
    assert torch.isnan(out[i, :G, 7]).all()
    assert torch.equal(torch.isnan(out), torch.isnan(plain))
    ok(pa, c.pool)
    c.pool.close()
