"""Plain 64-bit definitions of the 8-bit cache (codes, scales, the cache write,
pages) and of the norms before it.  numpy only; no code of the library."""
import numpy as np
import torch

from ._ops import BS, D, rand16, rope64

TOP = {"e4m3": 448.0, "int8": 127.0}
KINDS = ("e4m3", "int8")


def type8(kind):
    return torch.float8_e4m3fn if kind == "e4m3" else torch.int8


def _e4m3_values():
    v = np.zeros(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        x = np.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[b] = -x if b & 128 else x
    return v


E4M3 = _e4m3_values()


def decode8(codes, kind):
    """Bytes (uint8) -> what they stand for at scale 1."""
    return E4M3[codes] if kind == "e4m3" else codes.view(np.int8).astype(np.float64)


def encode8(x, kind):
    """The bytes nearest to x (|x| <= TOP), ties to the even code."""
    x = np.asarray(x, np.float64)
    if kind == "int8":
        return np.rint(x).astype(np.int8).view(np.uint8)
    pos = E4M3[:127]  # ascending, codes 0 .. 126
    a = np.abs(x)
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    down, up = a - pos[lo], pos[hi] - a
    c = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return (c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def need8(amax, kind):
    """Biased exponent of the smallest power of two >= 2^-126 whose largest code holds amax; 255 if it is not finite."""
    if not np.isfinite(amax):
        return 255
    x = -126
    if amax > TOP[kind] * 2.0 ** x:
        x = int(np.floor(np.log2(amax / TOP[kind]))) - 1
        while TOP[kind] * 2.0 ** x < amax:
            x += 1
        x = max(x, -126)
    return x + 127


def scale8(e):
    e = np.asarray(e, np.int64)
    return np.where(e == 255, np.nan, 2.0 ** (e - 127.0))


def runs_of(slots, n_slots):
    """The runs of a call: lists of consecutive rows whose slots follow each other inside one block."""
    runs, prev = [], None
    for r, s in enumerate(slots):
        if s < 0 or s >= n_slots:
            prev = None
            continue
        if prev is not None and s == prev + 1 and s % BS:
            runs[-1].append(r)
        else:
            runs.append([r])
        prev = s
    return runs


def write8(codes, exps, rows, slots, kind):
    """codes uint8 [N][H][16][128] and exps uint8 [N][H] after the write of rows [n][H][128] (float64)."""
    codes, exps = codes.copy(), exps.copy()
    N, H = exps.shape
    for run in runs_of(slots, N * BS):
        b, off = int(slots[run[0]]) // BS, int(slots[run[0]]) % BS
        at = off + np.arange(len(run))
        other = np.setdiff1d(np.arange(BS), at)
        for h in range(H):
            x = rows[run, h]
            e = need8(np.abs(x).max() if np.isfinite(x).all() else np.inf, kind)
            was = int(exps[b, h])
            if off and was >= e:
                e = was
            if off and e > was and e != 255:
                codes[b, h, other] = encode8(decode8(codes[b, h, other], kind) * 2.0 ** (was - e), kind)
            exps[b, h] = e
            if e != 255:
                codes[b, h, at] = encode8(x / 2.0 ** (e - 127.0), kind)
    return codes, exps


def norm64(x, w, eps):
    x = np.asarray(x, np.float64)
    if w is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def norm_rope64(x, w, eps, positions, inv_freq, axes, interleaved):
    return rope64(norm64(x, w, eps), positions, inv_freq, axes, interleaved)


def bytes_of(t):
    return t.detach().contiguous().view(torch.uint8).cpu().numpy()


def raw(pool):
    """Codes and exponents of a Pool8 as numpy: k, v, ek, ev."""
    return [bytes_of(t) for t in (pool.k, pool.v, pool.k_scale, pool.v_scale)]


def fill8(pool, k, v, ek, ev):
    for t, x in ((pool.k, k), (pool.v, v)):
        t.copy_(torch.from_numpy(x).cuda().view(pool.dtype))
    for t, x in ((pool.k_scale, ek), (pool.v_scale, ev)):
        t.copy_(torch.from_numpy(x).cuda().view(torch.float8_e8m0fnu))


def random8(rng, kind, n_blocks, hkv, spread=2):
    """Codes of normal rows and exponents that vary by block and head: [N][H][16][128], [N][H]."""
    x = rng.standard_normal((n_blocks, hkv, BS, D))
    top = np.abs(x).max((2, 3), keepdims=True)
    codes = encode8(x / top * TOP[kind], kind)
    exps = (127 + rng.integers(-spread, spread + 1, (n_blocks, hkv)) + (-7 if kind == "e4m3" else -5)).astype(np.uint8)
    return codes, exps


def filled_pool8(pa, rng, kind, n_blocks, hkv, spread=2):
    pool = pa.Pool8(n_blocks, hkv, type8(kind))
    k, ek = random8(rng, kind, n_blocks, hkv, spread)
    v, ev = random8(rng, kind, n_blocks, hkv, spread)
    fill8(pool, k, v, ek, ev)
    return pool, (k, v, ek, ev)


def values8(codes, exps, kind):
    return decode8(codes, kind) * scale8(exps)[..., None, None]


def ok8(pa, pool):
    code, detail = pa.pa_check8(pool)
    assert code == pa.PA_OK, (pa.strerror(code), detail)


def rand_rows(rng, dtype, n, h):
    return rand16(rng, dtype, n, h, D).cuda()
