"""Decode with attention-weight sums against its 64-bit definition.

Tolerance of a sum, from the arithmetic: a score is a 128-term product sum of
16-bit values in fp32, off by at most 128 * 2^-23 of sum |k q| * scale (the
tensor core may truncate each addition), plus two roundings of the score (2^-23
of its size); the log-sum-exp is off by as much again and by 2^-21 of itself;
exp turns absolute into relative error.  With sum |k q| * scale <= A the
weight is off by less than (2 * 128 * 2^-23 * A + 2^-20 (1 + |s|)) of itself."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, attend64, cache_rows, cuda, filled_pool, ok, rand16, tables_for, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


def tolerance(q, k, scale):
    """Largest relative error of a weight (natural-log units of the score)."""
    Hkv = k.shape[0]
    if k.shape[1] == 0:
        return 0.0
    a = float(np.einsum("hgd,htd->hgt", np.abs(q).reshape(Hkv, -1, D), np.abs(k)).max()) * abs(scale)
    return 2 * 128 * 2.0 ** -23 * a + 2.0 ** -20 * (1 + a)


CASES = [  # lens, Hq, Hkv, dtype, out, decay
    ([0, 1, 15, 16, 17, 100], 8, 2, torch.bfloat16, torch.float32, 1.0),
    ([513, 7, 256], 12, 2, torch.float16, torch.float16, 0.5),
    ([2049, 33], 5, 5, torch.float16, torch.float32, 0.0),
    ([300, 1000], 8, 1, torch.bfloat16, torch.bfloat16, 1.0),
    ([64, 5000], 21, 7, torch.bfloat16, torch.float32, 0.9375),
    ([40, 41], 10, 2, torch.float16, torch.float32, 1.0),
    ([9000], 7, 1, torch.bfloat16, torch.float32, 1.0),
    ([31] * 40, 32, 8, torch.bfloat16, torch.float32, 1.0),
    ([50, 20], 6, 1, torch.bfloat16, torch.float32, 1.0),
]


@pytest.mark.parametrize("lens,Hq,Hkv,dtype,out_dtype,decay", CASES)
def test_against_the_definition(pa, lens, Hq, Hkv, dtype, out_dtype, decay):
    rng = np.random.default_rng(sum(lens) + Hq)
    W = -(-max(lens) // BS) + 2
    tables, _, nb = tables_for(lens, rng, width=W)
    pool = filled_pool(pa, rng, nb, Hkv, dtype)
    B, scale = len(lens), 1 / np.sqrt(D)
    q = rand16(rng, dtype, B, Hq, D)
    w0 = rng.random((B, Hkv, W * BS)).astype(np.float32)
    w = cuda(w0)
    out = torch.full((B, Hq, D), float("nan"), dtype=out_dtype, device="cuda")
    bt, sl = cuda(tables), cuda(np.array(lens, np.int32))
    pa.pa_decode_weights(pool, q.cuda(), bt, sl, scale, out, w, decay=decay)
    ok(pa, pool)
    plain = torch.empty_like(out)
    pa.pa_decode_split(pool, q.cuda(), bt, sl, scale, plain)
    assert torch.equal(out, plain), "the output is the split decode's, bit for bit"
    k64, v64, q64, got = to64(pool.k), to64(pool.v), to64(q), w.cpu().numpy()
    for i, L in enumerate(lens):
        k = cache_rows(k64, tables[i], L)
        _, p = attend64(q64[i], k, cache_rows(v64, tables[i], L), scale)
        grown = p.reshape(Hkv, Hq // Hkv, L).sum(1)
        want = decay * w0[i, :, :L].astype(np.float64) + grown
        tol = tolerance(q64[i], k, scale) * grown + 2.0 ** -23 * (want + grown)  # (the sum and the last rounding)
        assert (np.abs(got[i, :, :L] - want) <= tol).all(), (i, np.abs(got[i, :, :L] - want).max())
        assert np.array_equal(got[i, :, L:], w0[i, :, L:]), "sums past the end untouched"
        if L:
            assert np.allclose(grown.sum(1), Hq // Hkv)
    pool.close()


def test_large_scores_and_a_workspace_kept(pa):
    """Scores of hundreds: one token takes everything; two calls with one
    workspace add up; NaN in slots past the end stays out."""
    rng = np.random.default_rng(9)
    lens, Hq, Hkv, dtype = [70, 19], 4, 1, torch.bfloat16
    tables, _, nb = tables_for(lens, rng)
    pool = filled_pool(pa, rng, nb, Hkv, dtype)
    pool.k.mul_(30.0)
    for i, L in enumerate(lens):  # slots past the end
        if L % BS:
            pool.k[tables[i, L // BS], :, L % BS:] = float("nan")
            pool.v[tables[i, L // BS], :, L % BS:] = float("nan")
    q = rand16(rng, dtype, 2, Hq, D).cuda()
    bt, sl = cuda(tables), cuda(np.array(lens, np.int32))
    w = torch.zeros(2, Hkv, tables.shape[1] * BS, device="cuda")
    out = torch.empty(2, Hq, D, device="cuda")
    ws = pa.weights_workspace_for(pool, q, bt)
    for _ in range(2):
        pa.pa_decode_weights(pool, q, bt, sl, 1.0, out, w, workspace=ws)
    ok(pa, pool)
    assert torch.isfinite(w).all() and torch.isfinite(out).all()
    for i, L in enumerate(lens):
        _, p = attend64(to64(q)[i], cache_rows(to64(pool.k), tables[i], L), cache_rows(to64(pool.v), tables[i], L), 1.0)
        want = 2 * p.sum(0)
        got = to64(w)[i, 0, :L]
        tol = tolerance(to64(q)[i], cache_rows(to64(pool.k), tables[i], L), 1.0)
        assert (np.abs(got - want) <= 2 * tol * np.maximum(want, 2.0 ** -100) + 2.0 ** -22 * want).all()
    pool.close()


def test_blocks_out_of_range_take_no_weight(pa):
    rng = np.random.default_rng(10)
    tables, _, nb = tables_for([48, 20], rng)
    pool = filled_pool(pa, rng, nb, 2, torch.float16)
    q = rand16(rng, torch.float16, 2, 4, D).cuda()
    bad = tables.copy()
    bad[0, 1] = nb
    bad[1] = -3
    w = torch.zeros(2, 2, 48, device="cuda")
    out = torch.empty(2, 4, D, device="cuda")
    pa.pa_decode_weights(pool, q, cuda(bad), cuda(np.array([48, 20], np.int32)), 0.1, out, w)
    assert pa.pa_check(pool)[0] == pa.PA_ERR_DEVICE_CHECK
    assert (w[0, :, 16:32] == 0).all() and (w[1] == 0).all()
    assert torch.allclose(w[0].sum(1), torch.full((2,), 2.0, device="cuda"), atol=1e-5)
    pool.close()


def test_graph_replay_and_other_stream(pa):
    rng = np.random.default_rng(11)
    lens, Hq, Hkv, dtype = [700, 90, 1], 8, 2, torch.bfloat16
    tables, _, nb = tables_for(lens, rng)
    pool = filled_pool(pa, rng, nb, Hkv, dtype)
    q = rand16(rng, dtype, 3, Hq, D).cuda()
    bt, sl = cuda(tables), cuda(np.array(lens, np.int32))
    w = torch.zeros(3, Hkv, tables.shape[1] * BS, device="cuda")
    out, ref = torch.empty(3, Hq, D, device="cuda"), torch.empty(3, Hq, D, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pa.pa_decode_weights(pool, q, bt, sl, 0.1, ref, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    one = w.clone()
    w.zero_()
    ws = pa.weights_workspace_for(pool, q, bt)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_decode_weights(pool, q, bt, sl, 0.1, out, w, workspace=ws)
    g.replay()
    assert torch.equal(w, one) and torch.equal(out, ref)
    g.replay()
    assert torch.allclose(w, 2 * one)
    ok(pa, pool)
    pool.close()


def test_refusals(pa):
    pool = pa.Pool(4, 2, torch.bfloat16)
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    good = dict(q=z(2, 4, D, t=torch.bfloat16), block_tables=z(2, 2), seq_lens=z(2), scale=0.1,
                out=z(2, 4, D, t=torch.float32), weights=z(2, 2, 32, t=torch.float32))
    pa.pa_decode_weights(pool, **good)
    for change, error in [(dict(weights=z(2, 2, 31, t=torch.float32)), ValueError),
                          (dict(weights=z(2, 2, 32, t=torch.float64)), TypeError),
                          (dict(weights=z(2, 4, 32, t=torch.float32)[:, ::2]), ValueError),
                          (dict(weights=z(2 * 2 * 32 + 1, t=torch.float32)[1:].view(2, 2, 32)), pa.PagedAttentionError),
                          (dict(q=z(2, 18, D, t=torch.bfloat16), out=z(2, 18, D, t=torch.float32)), pa.PagedAttentionError),
                          (dict(q=z(2, 3, D, t=torch.bfloat16), out=z(2, 3, D, t=torch.float32)), pa.PagedAttentionError),
                          (dict(workspace=z(64, t=torch.uint8)), pa.PagedAttentionError)]:
        with pytest.raises(error):
            pa.pa_decode_weights(pool, **{**good, **change})
    ok(pa, pool)
    pool.close()
