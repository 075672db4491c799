"""Pages between a 16-bit and an 8-bit pool, byte for byte against the
definition: scaling by powers of two is exact, each way rounds once."""
import numpy as np
import pytest
import torch

from ._ops import BS, cuda, filled_pool, to64
from ._ops8 import KINDS, encode8, fill8, filled_pool8, need8, ok8, raw, scale8, type8, values8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


def i32(x):
    return cuda(np.asarray(x, np.int32))


def bits16(t):
    return t.view(torch.int16).cpu().numpy()


def quantized(x, codes, exps, src, dst, rows, kind):
    """x [N][H][16][128] float64 into copies of codes and exps."""
    codes, exps = codes.copy(), exps.copy()
    for a, b, n in zip(src, dst, rows):
        for h in range(x.shape[1]):
            t = x[a, h, :n]
            e = need8(np.abs(t).max(initial=0.0) if np.isfinite(t).all() else np.inf, kind)
            exps[b, h] = e
            if e != 255:
                codes[b, h, :n] = encode8(t / scale8(e), kind)
    return codes, exps


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hkv,n", [(1, 1), (2, 9), (5, 40), (8, 333)])
def test_there_and_back(pa, kind, dtype, hkv, n):
    rng = np.random.default_rng(n + hkv)
    N, N8 = 2 * n + 1, n + 2
    pool = filled_pool(pa, rng, N, hkv, dtype)
    size = torch.from_numpy(2.0 ** rng.integers(-9, 9, (2, N, hkv, 1, 1)).astype(np.float32)).to(dtype).cuda()
    pool.k.mul_(size[0]), pool.v.mul_(size[1])
    pool8, (k, v, ek, ev) = filled_pool8(pa, rng, kind, N8, hkv)
    perm = rng.permutation(N)
    src, back, dst = perm[:n], perm[n:2 * n], rng.permutation(N8)[:n]
    rows = rng.integers(0, BS + 1, n)
    rows[: n // 2] = BS
    k16, v16 = to64(pool.k), to64(pool.v)
    pa.pa_quantize_blocks(pool, i32(src), pool8, i32(dst), rows=i32(rows))
    k, ek = quantized(k16, k, ek, src, dst, rows, kind)
    v, ev = quantized(v16, v, ev, src, dst, rows, kind)
    for got, ref in zip(raw(pool8), (k, v, ek, ev)):
        assert np.array_equal(got, ref)
    pa.pa_dequantize_blocks(pool8, i32(dst), pool, i32(back))
    for t, x, codes, exps in ((pool.k, k16, k, ek), (pool.v, v16, v, ev)):
        val = torch.from_numpy(values8(codes, exps, kind)[dst])
        x = x.copy()
        x[back] = val.to(dtype).double().numpy()
        assert np.array_equal(to64(t), x)
    ok8(pa, pool8)


@pytest.mark.parametrize("kind", KINDS)
def test_without_rows_all_sixteen_count(pa, kind):
    rng = np.random.default_rng(3)
    pool = filled_pool(pa, rng, 5, 3, torch.bfloat16)
    a, b = pa.Pool8(5, 3, type8(kind)), pa.Pool8(5, 3, type8(kind))
    ids = i32(rng.permutation(5))
    pa.pa_quantize_blocks(pool, ids, a, ids)
    pa.pa_quantize_blocks(pool, ids, b, ids, rows=i32([16] * 5))
    for x, y in zip(raw(a), raw(b)):
        assert np.array_equal(x, y) and x.any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_not_finite_and_largest_values(pa, kind, dtype):
    top = torch.finfo(dtype).max
    pool = pa.Pool(4, 1, dtype)
    pool.k[0, 0, 3, 7], pool.k[1, 0, 15, 127], pool.v[0, 0, 0, 0] = float("nan"), float("-inf"), float("inf")
    pool.v[1].fill_(top)
    pool.v[1, 0, 0] = -top
    pool8 = pa.Pool8(2, 1, type8(kind))
    ids = i32([0, 1])
    pa.pa_quantize_blocks(pool, ids, pool8, ids, rows=i32([16, 15]))
    _, _, ek, ev = raw(pool8)
    assert ek[:, 0].tolist() == [255, 1] and ev[0, 0] == 255, "row 15 of block 1 does not count"
    pa.pa_dequantize_blocks(pool8, ids, pool, i32([2, 3]))
    assert torch.isnan(pool.k[2]).all() and torch.isnan(pool.v[2]).all()
    got = pool.v[3].float()
    assert torch.isfinite(got).all() and (got[0, 0] < 0).all() and (got[0, 1:15] > 0.98 * top).all(), "saturated"
    assert (got[0, 15] == 0).all()


def test_ids_and_rows_out_of_range(pa):
    rng = np.random.default_rng(4)
    pool = filled_pool(pa, rng, 4, 2, torch.bfloat16)
    pool8, state = filled_pool8(pa, rng, "int8", 4, 2)
    k16 = bits16(pool.k)
    for src, dst, detail in (([0, 4], [1, 2], 4), ([0, -1], [1, 2], -1), ([0, 1], [1, 4], 4), ([0, 1], [1, -7], -7)):
        fill8(pool8, *state)
        pa.pa_quantize_blocks(pool, i32(src), pool8, i32(dst))
        assert pa.pa_check8(pool8) == (pa.PA_ERR_DEVICE_CHECK, detail)
        got = raw(pool8)
        for x, y in zip(got, state):
            assert np.array_equal(np.delete(x, 1, 0), np.delete(y, 1, 0))
        # (block 1 is written; its exponents may be the ones it had)
        assert not np.array_equal(got[0][1], state[0][1]) and not np.array_equal(got[1][1], state[1][1])
        pa.pa_dequantize_blocks(pool8, i32(src[1:]), pool, i32(dst[1:]))
        assert pa.pa_check8(pool8) == (pa.PA_ERR_DEVICE_CHECK, detail)
        assert np.array_equal(bits16(pool.k), k16)
    for rows, as_if in ((17, 16), (-1, 0)):
        fill8(pool8, *state)
        pa.pa_quantize_blocks(pool, i32([2]), pool8, i32([3]), rows=i32([rows]))
        assert pa.pa_check8(pool8) == (pa.PA_ERR_DEVICE_CHECK, rows)
        got = raw(pool8)
        fill8(pool8, *state)
        pa.pa_quantize_blocks(pool, i32([2]), pool8, i32([3]), rows=i32([as_if]))
        for x, y in zip(got, raw(pool8)):
            assert np.array_equal(x, y)
        ok8(pa, pool8)


def test_copies_inside_the_pool(pa):
    rng = np.random.default_rng(5)
    pool, state = filled_pool8(pa, rng, "e4m3", 30, 5)
    perm = rng.permutation(30)
    src, dst = perm[:10], perm[10:20]
    pa.pa_copy_blocks8(pool, i32(src), i32(dst))
    ok8(pa, pool)
    for got, x in zip(raw(pool), state):
        x = x.copy()
        x[dst] = x[src]
        assert np.array_equal(got, x)
    pa.pa_copy_blocks8(pool, i32([30]), i32([0]))
    assert pa.pa_check8(pool) == (pa.PA_ERR_DEVICE_CHECK, 30)
    pa.pa_copy_blocks8(pool, i32([]), i32([]))


def test_pages_behind_four_gigabytes(pa):
    rng = np.random.default_rng(6)
    n = 150000
    pool16 = filled_pool(pa, rng, 6, 8, torch.bfloat16)
    small, big = pa.Pool8(6, 8, torch.int8), pa.Pool8(n, 8, torch.int8)
    ids, top = i32(range(6)), i32(range(n - 6, n))
    pa.pa_quantize_blocks(pool16, ids, small, ids)
    pa.pa_quantize_blocks(pool16, ids, big, top)
    assert torch.equal(big.k[n - 6:], small.k) and torch.equal(big.v[n - 6:], small.v)
    pa.pa_copy_blocks8(big, top, ids)
    assert torch.equal(big.v[:6], small.v)
    want = pa.Pool(6, 8, torch.bfloat16)
    pa.pa_dequantize_blocks(small, ids, want, ids)
    pa.pa_dequantize_blocks(big, top, pool16, ids)
    assert torch.equal(pool16.k, want.k) and torch.equal(pool16.v, want.v)
    ok8(pa, big)
    big.close()


def test_graph_and_stream(pa):
    rng = np.random.default_rng(7)
    pool = filled_pool(pa, rng, 8, 2, torch.float16)
    pool8 = pa.Pool8(4, 2, torch.float8_e4m3fn)
    ids, back = i32([0, 1, 2, 3]), i32([4, 5, 6, 7])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    pa.pa_quantize_blocks(pool, ids, pool8, ids, stream=st)
    pa.pa_dequantize_blocks(pool8, ids, pool, back, stream=st)
    st.synchronize()
    want = pool.k.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_quantize_blocks(pool, ids, pool8, ids)
        pa.pa_dequantize_blocks(pool8, ids, pool, back)
    pool.k[4:].zero_()
    pool8.k.view(torch.uint8).zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(pool.k, want)


def test_refusals(pa):
    pool, pool8 = pa.Pool(4, 2, torch.bfloat16), pa.Pool8(4, 3, torch.int8)
    ids = i32([0, 1])
    with pytest.raises(pa.PagedAttentionError):  # another number of heads
        pa.pa_quantize_blocks(pool, ids, pool8, ids)
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_dequantize_blocks(pool8, ids, pool, ids)
    with pytest.raises(TypeError):
        pa.pa_quantize_blocks(pool8, ids, pool, ids)
    pool8 = pa.Pool8(4, 2, torch.int8)
    with pytest.raises(ValueError):
        pa.pa_quantize_blocks(pool, ids, pool8, ids[:1])
    with pytest.raises(ValueError):
        pa.pa_quantize_blocks(pool, ids, pool8, ids, rows=ids[:1])
    with pytest.raises(TypeError):
        pa.pa_quantize_blocks(pool, ids.long(), pool8, ids)
    with pytest.raises(ValueError):
        pa.pa_copy_blocks8(pool8, ids, ids[:1])
    with pytest.raises(KeyError):
        pa.Pool8(4, 2, torch.bfloat16)
    with pytest.raises(pa.PagedAttentionError):
        pa.Pool8(4, 2, torch.int8, d_head=64)
    pa.pa_quantize_blocks(pool, ids[:0], pool8, ids[:0])
