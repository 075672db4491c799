"""Eviction against its definition: positions, rows, sums and lengths are exact."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, cuda, evict64, filled_pool, ok, tables_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


def bits(t):
    return t.detach().cpu().view(torch.int16).numpy()


def weights_of(rng, kind, shape):
    w = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        w = np.round(w).astype(np.float32)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "odd":  # what the type can hold
        pick = rng.integers(0, 9, shape)
        for k, x in enumerate([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -3.5, np.finfo(np.float32).max]):
            w[pick == k] = x
    return w


def run_and_check(pa, lens, keep, n_sink, n_recent, hkv, dtype, kind, place, seed=0, extra_width=0):
    rng = np.random.default_rng(seed)
    wide = max(-(-int(max(lens)) // BS), 1) + extra_width
    n_of = [min(k, L) for k, L in zip(keep, lens)]
    wd = max(1, max(-(-n // BS) for n in n_of)) + (1 if place == "fresh" else 0)
    tables, free, nb = tables_for(lens, rng, spare=len(lens) * wd + 2, width=wide)
    pool = filled_pool(pa, rng, nb, hkv, dtype)
    k0, v0 = bits(pool.k).copy(), bits(pool.v).copy()
    w = weights_of(rng, kind, (len(lens), hkv, wide * BS))
    if place == "in place":
        dst = None
    else:
        dst = free[:len(lens) * wd].reshape(len(lens), wd).copy()
        if place == "mixed":  # every other block stays in place
            for i, L in enumerate(lens):
                for j in range(0, min(wd, -(-L // BS)), 2):
                    dst[i, j] = tables[i, j]
    kept = torch.full((len(lens), hkv, wide * BS), -7, dtype=torch.int32, device="cuda")
    wt = cuda(w)
    out = wt if place == "in place" else torch.full_like(wt, -5.0)
    lens_out = torch.full((len(lens),), -1, dtype=torch.int32, device="cuda")
    pa.pa_evict(pool, wt, cuda(tables), cuda(np.array(lens, np.int32)), cuda(np.array(keep, np.int32)), lens_out, kept,
                n_sink=n_sink, n_recent=n_recent, dst_tables=None if dst is None else cuda(dst), weights_out=out)
    ok(pa, pool)
    assert lens_out.cpu().tolist() == n_of
    k1, v1 = k0.copy(), v0.copy()
    w1 = w.copy() if place == "in place" else np.full_like(w, -5.0)
    kept1 = np.full(kept.shape, -7, np.int32)
    d = tables if dst is None else dst
    for i, L in enumerate(lens):
        for h in range(hkv):
            at = evict64(w[i, h], L, keep[i], n_sink, n_recent)
            n, j = len(at), np.arange(len(at))
            kept1[i, h, :n] = at
            w1[i, h, :n] = w[i, h, at]
            w1[i, h, n:L] = 0
            for x1, x0 in ((k1, k0), (v1, v0)):
                x1[d[i, j // BS], h, j % BS] = x0[tables[i, at // BS], h, at % BS]
    assert np.array_equal(kept.cpu().numpy(), kept1), "kept positions"
    assert np.array_equal(out.cpu().numpy().view(np.int32), w1.view(np.int32)), "weight sums"
    assert np.array_equal(bits(pool.k), k1) and np.array_equal(bits(pool.v), v1), "rows"
    if place != "in place":
        assert np.array_equal(wt.cpu().numpy().view(np.int32), w.view(np.int32))
    pool.close()


@pytest.mark.parametrize("place", ["in place", "fresh", "mixed"])
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
def test_ragged_lengths(pa, place, kind):
    lens = [0, 1, 2, 15, 16, 17, 33, 300, 1023, 1024, 1025, 2500]
    keep = [5, 1, 1, 15, 8, 16, 0, 77, 1000, 512, 1025, 100]
    run_and_check(pa, lens, keep, 4, 8, 3, torch.bfloat16, kind, place, seed=1, extra_width=3)


@pytest.mark.parametrize("n_sink,n_recent", [(0, 0), (1, 0), (0, 1), (5, 300), (300, 5), (1 << 30, 1 << 30)])
def test_protected_ends(pa, n_sink, n_recent):
    run_and_check(pa, [1, 10, 200, 517], [1, 4, 60, 400], n_sink, n_recent, 2, torch.float16, "ties", "in place", seed=2)


@pytest.mark.parametrize("place", ["in place", "fresh"])
def test_long_sequence_many_ratios(pa, place):
    run_and_check(pa, [70001], [333], 16, 64, 1, torch.float16, "plain", place, seed=3)
    run_and_check(pa, [40000, 39999], [39990, 20001], 4, 64, 2, torch.bfloat16, "ties", place, seed=4)


def test_one_kv_head_per_query_head_layout(pa):
    run_and_check(pa, [600, 64, 129], [128, 64, 128], 4, 16, 40, torch.float16, "plain", "in place", seed=5)


def test_device_checks(pa):
    """Out-of-range lengths, keeps and blocks are reported, clamped or skipped; nothing else changes."""
    rng = np.random.default_rng(7)
    tables, free, nb = tables_for([40, 40], rng)
    pool = filled_pool(pa, rng, nb, 1, torch.bfloat16)
    w = cuda(np.ones((2, 1, 48), np.float32))
    kept = torch.zeros(2, 1, 48, dtype=torch.int32, device="cuda")
    n_out = torch.zeros(2, dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    call = lambda t, L, n, **kw: pa.pa_evict(pool, w.clone(), t, L, n, n_out, kept, **kw)  # noqa: E731
    t = cuda(tables)
    call(t, i32(49, 40), i32(10, 10))
    assert pa.pa_check(pool) == (pa.PA_ERR_DEVICE_CHECK, 49) and n_out.tolist() == [10, 10]
    call(t, i32(40, 40), i32(-3, 10))
    assert pa.pa_check(pool) == (pa.PA_ERR_DEVICE_CHECK, -3) and n_out.tolist() == [0, 10]
    call(t, i32(40, 40), i32(33, 10), dst_tables=cuda(free[:2].reshape(2, 1)))
    assert pa.pa_check(pool) == (pa.PA_ERR_DEVICE_CHECK, 33) and n_out.tolist() == [16, 10]
    k0 = pool.k.clone()
    bad = tables.copy()
    bad[0] = nb
    call(cuda(bad), i32(40, 0), i32(10, 10))
    assert pa.pa_check(pool)[0] == pa.PA_ERR_DEVICE_CHECK
    assert torch.equal(k0.view(torch.int16), pool.k.view(torch.int16))
    pool.close()


def test_refusals(pa):
    pool = pa.Pool(4, 2, torch.bfloat16)
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    good = dict(weights=z(3, 2, 32, t=torch.float32), block_tables=z(3, 2), seq_lens=z(3), keep=z(3), seq_lens_out=z(3),
                kept=z(3, 2, 32))
    pa.pa_evict(pool, **good)
    lens = z(3)
    for change, error in [(dict(weights=z(3, 2, 31, t=torch.float32)), ValueError), (dict(weights=z(3, 2, 32)), TypeError),
                          (dict(kept=z(3, 2, 16)), ValueError), (dict(keep=z(2)), ValueError),
                          (dict(seq_lens=lens, seq_lens_out=lens), pa.PagedAttentionError),
                          (dict(keep=lens, seq_lens_out=lens), pa.PagedAttentionError),
                          (dict(n_sink=-1), pa.PagedAttentionError), (dict(n_recent=-1), pa.PagedAttentionError),
                          (dict(dst_tables=z(2, 2)), ValueError), (dict(dst_tables=z(3, 0)), pa.PagedAttentionError),
                          (dict(weights=torch.zeros(3, 2, 32)), ValueError)]:
        with pytest.raises(error):
            pa.pa_evict(pool, **{**good, **change})
    pa.pa_evict(pool, z(0, 2, 32, t=torch.float32), z(0, 2), z(0), z(0), z(0), z(0, 2, 32))
    ok(pa, pool)
    pool.close()
