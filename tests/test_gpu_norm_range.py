"""Norms over the whole range of their rows: squares that leave 32 bits at either end, with and without eps.

Tolerance: that of the norms' other tests, 2^-18 of |x| + |y| of the normed pair (scaling a row by a power of two is
exact while its numbers are normal).  Below 2^-126 a number of 32 bits is off by 2^-150 an operation, of which there are
fewer than 2^10 to an output of size 1: 2^-140, beside half a step (2^-134) of the smallest bf16 numbers."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, half_step, ok, to64
from ._ops8 import KINDS, decode8, need8, ok8, raw, scale8, type8
from .test_gpu_norm_rope import Tokens, pair_size, weight

pytestmark = pytest.mark.gpu
SIZES = [2.0 ** e for e in (-130, -120, -90, -76, -70, -55, -20, 0, 40, 59, 62, 64, 70, 100, 124)]
EPSES = [0.0, 2.0 ** -140, 1e-36, 1e-30, 1e-6, 1.0, 1e30, 3e38]


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


def tokens(rng, n, Hq, Hkv, dtype, sizes, rot=128, interleaved=False):
    """Rows of one size after the other: neighbours in a call differ."""
    t = Tokens(rng, n, Hq, Hkv, dtype, rot, 1, interleaved)
    for x in (t.q, t.k):
        x.copy_(torch.from_numpy(rng.standard_normal(x.shape)).clamp(-2.5, 2.5).cuda()
                * torch.tensor([[sizes[(3 * i + h) % len(sizes)]] for i in range(n) for h in range(x.shape[1])],
                               dtype=torch.float64, device="cuda").view(n, x.shape[1], 1))
    return t


def close(got, ref, normed, dtype, rot=128, interleaved=False):
    slack = 2.0 ** -18 * pair_size(normed, rot, interleaved) + 2.0 ** -140
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134
    bad = ~(np.abs(got - ref) <= half_step(dtype) * (np.abs(ref) + slack) + slack + tiny)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0].tolist(), got[bad][:3], ref[bad][:3])


@pytest.mark.parametrize("eps", EPSES)
@pytest.mark.parametrize("n,Hq,Hkv,interleaved,norms", [(9, 32, 8, False, "qk"), (500, 30, 3, True, "qk"), (500, 32, 8, False, "k")])
def test_rows_of_every_size(pa, eps, n, Hq, Hkv, interleaved, norms):
    rng = np.random.default_rng(n + Hq)
    eps = float(np.float32(eps))
    for dtype, sizes in ((torch.bfloat16, SIZES), (torch.float16, [2.0 ** -24, 2.0 ** -16, 1.0, 2.0 ** 14])):
        t = tokens(rng, n, Hq, Hkv, dtype, sizes, interleaved=interleaved)
        wq, wk = (weight(rng, dtype) if x in norms else None for x in "qk")
        pool = pa.Pool(-(-n // BS), Hkv, dtype)
        pa.pa_norm_rope_append(pool, *t.args(wq, wk, np.arange(n)), eps=eps, interleaved=interleaved)
        ok(pa, pool)
        rows = to64(pool.k).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:n]
        for got, x, w in ((to64(t.q_out), t.q, wq), (rows, t.k, wk)):
            with np.errstate(invalid="ignore"):
                ref, normed = t.want(x, w, eps)
            nothing = to64(x).any(-1) == 0  # (fp16 rows that rounded to zero: 0 / 0 without eps)
            if eps == 0.0 and w is not None:
                assert np.isnan(got[nothing]).all()
                got, ref, normed = got[~nothing], ref[~nothing], normed[~nothing]
            close(got, ref, normed, dtype, 128, interleaved)
        pool.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6, 3e38])
@pytest.mark.parametrize("n", [20, 1000])
def test_rows_of_every_size_into_8_bits(pa, kind, eps, n):
    """Each token starts a block, so that its row alone sets the scale."""
    rng = np.random.default_rng(n)
    eps = float(np.float32(eps))
    dtype, Hkv = torch.bfloat16, 2
    t = tokens(rng, n, 8, Hkv, dtype, SIZES)
    w = weight(rng, dtype)
    pool = pa.Pool8(n, Hkv, type8(kind))
    pa.pa_norm_rope_append8(pool, *t.args(w, w, np.arange(n) * BS), eps=eps)
    ok8(pa, pool)
    ref, normed = t.want(t.q, w, eps)
    close(to64(t.q_out), ref, normed, dtype)
    ref, normed = t.want(t.k, w, eps)
    slack = 2.0 ** -18 * pair_size(normed, 128, False) + 2.0 ** -140
    k, _, ek, _ = raw(pool)
    for h in range(Hkv):
        x, d = ref[:, h], slack[:, h]
        for i in range(n):
            assert int(ek[i, h]) in {need8(a, kind) for a in (max((np.abs(x[i]) - d[i]).max(), 0), (np.abs(x[i]) + d[i]).max())}
        s = scale8(ek[:, h])[:, None]
        step = s + 0 * x if kind == "int8" else s * 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x) / s, 2.0 ** -6))) - 3)
        assert (np.abs(decode8(k[:, h, 0], kind) * s - x) <= step / 2 * (1 + 2.0 ** -10) + d).all()


def test_rows_that_are_not_finite_or_zero(pa):
    """x / sqrt(mean(x^2) + eps) as it stands: a row with an infinity is zero elsewhere and NaN there (its pair after the
    rotation, too), a row with a NaN is NaN, a row of zeros without eps too; their neighbours do not change."""
    rng = np.random.default_rng(5)
    dtype = torch.bfloat16
    t = tokens(rng, 6, 8, 2, dtype, SIZES)
    w = weight(rng, dtype)
    pool = pa.Pool(1, 2, dtype)
    pa.pa_norm_rope_append(pool, *t.args(w, w, np.arange(6)), eps=0.0)
    clean = t.q_out.clone()
    t.q[1, 2], t.q[2, 3, 7], t.q[4, 0, 100] = 0.0, float("nan"), float("-inf")
    t.q_out.fill_(1.0)
    pa.pa_norm_rope_append(pool, *t.args(w, w, np.arange(6)), eps=0.0)
    assert torch.isnan(t.q_out[1, 2]).all() and torch.isnan(t.q_out[2, 3]).all()
    pair = torch.tensor([36, 100], device="cuda")
    assert torch.isnan(t.q_out[4, 0, pair]).all()
    rest = torch.ones(D, dtype=torch.bool, device="cuda")
    rest[pair] = False
    assert (t.q_out[4, 0, rest] == 0).all()
    for i, h in ((1, 2), (2, 3), (4, 0)):
        t.q_out[i, h] = clean[i, h]
    assert torch.equal(t.q_out, clean)


@pytest.mark.parametrize("n", [40, 1200])
def test_a_row_out_of_range_leaves_its_neighbours_alone(pa, n):
    """Rows that share a warp with one that has to be scaled keep their bits."""
    rng = np.random.default_rng(8)
    dtype = torch.bfloat16
    t = tokens(rng, n, 8, 3, dtype, [1.0])
    w = weight(rng, dtype)
    results = []
    for _ in range(2):
        p8, p16 = pa.Pool8(n, 3, type8("e4m3")), pa.Pool(n, 3, dtype)
        pa.pa_norm_rope_append8(p8, *t.args(w, w, np.arange(n) * BS))
        q = t.q_out.clone()
        pa.pa_norm_rope_append(p16, *t.args(w, w, np.arange(n) * BS))
        assert torch.equal(q, t.q_out)
        results.append((raw(p8), p16.k.clone(), q))
        t.k[3, 1] *= 2.0 ** 80
        t.q[7, 5] *= 2.0 ** -90
    (a, ka, qa), (b, kb, qb) = results
    for x in (a, b):
        for y in x:
            y[3, 1] = 0
    for x, y in zip(a, b):
        assert np.array_equal(x, y)
    ka[3, 1], kb[3, 1] = 0.0, 0.0
    qa[7, 5], qb[7, 5] = 0.0, 0.0
    assert torch.equal(ka, kb) and torch.equal(qa, qb)
