"""NaN in the cache reaches every row that attends it, also where the row's
tokens are joined from parts: softmax over a NaN score is NaN everywhere, and a
weight of zero times a NaN value is NaN."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, cuda, filled_pool, ok, rand16, tables_for
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


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (7, 1)])
@pytest.mark.parametrize("blocks", [0, 3, 100, 300, 301, 302, 303, 304, 305, 306, 307, 308])
def test_weight_sums_behind_a_nan_key(pa, blocks, Hq, Hkv):
    """The NaN key is the only token of the sequence's last tile, which, for
    some of the lengths, is the only tile of the last range: every token of the
    sequence then has a NaN weight, as where the sequence is not cut."""
    L = blocks * BS + 1
    rng = np.random.default_rng(blocks)
    tables, _, nb = tables_for([L, 50], rng)
    pool = filled_pool(pa, rng, nb, Hkv, torch.bfloat16)
    pool.k[int(tables[0, blocks]), Hkv - 1, 0, 3] = float("nan")
    q = rand16(rng, torch.bfloat16, 2, Hq, D).cuda()
    w = torch.zeros(2, Hkv, tables.shape[1] * BS, device="cuda")
    out = torch.empty(2, Hq, D, device="cuda")
    pa.pa_decode_weights(pool, q, cuda(tables), cuda(np.array([L, 50], np.int32)), D ** -0.5, out, w)
    ok(pa, pool)
    G = Hq // Hkv
    assert torch.isnan(out[0, (Hkv - 1) * G:]).all() and torch.isfinite(out[0, :(Hkv - 1) * G]).all()
    assert torch.isnan(w[0, Hkv - 1, :L]).all() and torch.isfinite(w[0, :Hkv - 1]).all()
    assert (w[0, :, L:] == 0).all() and torch.isfinite(w[1]).all() and torch.isfinite(out[1]).all()
    pool.close()


@pytest.mark.parametrize("which", ["first", "last"])
def test_weight_sums_where_most_of_the_keys_are_nan(pa, which):
    """More than 32 ranges of one sequence without a finite score, before or behind the others."""
    L, Hkv = 9000, 1
    tables, _, nb = tables_for([L], np.random.default_rng(1))
    pool = filled_pool(pa, np.random.default_rng(2), nb, Hkv, torch.bfloat16)
    at = torch.from_numpy(tables[0].astype(np.int64)).cuda()
    pool.k[at[:-60] if which == "first" else at[60:]] = float("nan")
    q = rand16(np.random.default_rng(3), torch.bfloat16, 1, 4, D).cuda()
    w = torch.zeros(1, Hkv, tables.shape[1] * BS, device="cuda")
    out = torch.empty(1, 4, D, device="cuda")
    pa.pa_decode_weights(pool, q, cuda(tables), cuda(np.array([L], np.int32)), D ** -0.5, out, w)
    ok(pa, pool)
    assert torch.isnan(w[0, 0, :L]).all() and (w[0, 0, L:] == 0).all()
    pool.close()
