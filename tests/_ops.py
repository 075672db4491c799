"""Plain 64-bit definitions of the cache operators (rotary append, decode with
weight sums, eviction, shared-prefix decode) and small input makers for their
tests.  numpy only; no code of the library."""
import numpy as np
import torch

BS, D = 16, 128


def to64(t):
    return t.detach().cpu().double().numpy()


def rope64(x, positions, inv_freq, axis_of_pair, interleaved):
    """x [n][h][128]; positions int [axes][n]; returns the turned rows."""
    rot = 2 * len(inv_freq)
    a = np.stack([positions[ax] for ax in axis_of_pair], 1).astype(np.float64) * np.asarray(inv_freq, np.float64)
    c, s = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
    i = np.arange(rot // 2)
    i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y = np.array(x, np.float64)
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    return y


def cache_rows(pool, table, L):
    """The first L rows of a sequence's cache, [h][L][128] (pool: numpy [N][h][16][128])."""
    nb = -(-L // BS)
    x = pool[np.asarray(table[:nb], np.int64)].transpose(1, 0, 2, 3)
    return x.reshape(x.shape[0], nb * BS, D)[:, :L]


def attend64(q, k, v, scale):
    """q [Hq][128], k and v [Hkv][L][128] -> out [Hq][128], softmax [Hq][L]."""
    Hkv, L, _ = k.shape
    G = q.shape[0] // Hkv
    if L == 0:
        return np.zeros_like(q), np.zeros((q.shape[0], 0))
    s = np.einsum("hgd,htd->hgt", q.reshape(Hkv, G, D), k) * scale
    s = np.exp(s - s.max(2, keepdims=True))
    p = s / s.sum(2, keepdims=True)
    return np.einsum("hgt,htd->hgd", p, v).reshape(-1, D), p.reshape(-1, L)


def evict64(w, L, keep, n_sink, n_recent):
    """The kept positions of one kv head, ascending; w float32 [>= L]."""
    n = min(keep, L)
    a = min(n_sink, n)
    b = min(n_recent, n - a)
    mid = w[a:L - b].astype(np.float64)
    mid = np.where(np.isnan(mid), -np.inf, mid)
    nan = np.isnan(w[a:L - b])
    order = np.lexsort((np.arange(len(mid)), nan, -mid))  # by weight, NaN behind -inf, then position
    mid = np.sort(order[:n - a - b]) + a
    return np.concatenate([np.arange(a), mid, np.arange(L - b, L)]).astype(np.int64)


def tables_for(lens, rng, spare=4, width=None):
    """Block tables [B][W] (-1 past the end) at random places, the free blocks, the pool's size."""
    nb = [-(-int(L) // BS) for L in lens]
    n = sum(nb) + spare
    perm = rng.permutation(n).astype(np.int32)
    W = max(max(nb), 1) if width is None else width
    t = np.full((len(lens), W), -1, np.int32)
    at = 0
    for i, k in enumerate(nb):
        t[i, :k] = perm[at:at + k]
        at += k
    return t, perm[at:], n


def rand16(rng, dtype, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)


def filled_pool(pa, rng, n_blocks, hkv, dtype):
    pool = pa.Pool(n_blocks, hkv, dtype)
    pool.k.copy_(rand16(rng, dtype, n_blocks, hkv, BS, D))
    pool.v.copy_(rand16(rng, dtype, n_blocks, hkv, BS, D))
    return pool


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def half_step(dtype):
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def ok(pa, pool):
    code, detail = pa.pa_check(pool)
    assert code == pa.PA_OK, (pa.strerror(code), detail)
