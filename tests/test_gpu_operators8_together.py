"""The 8-bit cache as a serving loop uses it: prompts written in chunks, decode
steps, a fork with copy on write, a request parked in 8 bits and brought back
into a 16-bit pool; compared with a history in 64 bits that keeps the codes."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, attend64, cache_rows, cuda, filled_pool, ok, to64
from ._ops8 import KINDS, ok8, raw, type8, values8
from .test_gpu_norm_rope import Tokens, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,Hq,Hkv", [(torch.bfloat16, 8, 2), (torch.float16, 6, 3)])
def test_a_serving_history(pa, kind, dtype, Hq, Hkv):
    rng = np.random.default_rng(1)
    n_blocks = 64
    pool = pa.Pool8(n_blocks, Hkv, type8(kind))
    alloc = pa.BlockAllocator(n_blocks, free_order=rng.permutation(n_blocks))
    wq, wk = weight(rng, dtype), weight(rng, dtype)
    rows = {}     # sequence -> its K and V rows in 64 bits, [token][Hkv][128]

    def step(counts):
        """counts: {sequence: new tokens}; one call for all of them, then one decode."""
        slots, who = [], []
        for s, n in counts.items():
            got, (a, b) = alloc.extend(s, n)
            if a >= 0:
                pa.pa_copy_blocks8(pool, cuda(np.array([a], np.int32)), cuda(np.array([b], np.int32)))
            slots += got.tolist()
            who += [s] * n
        t = Tokens(rng, len(slots), Hq, Hkv, dtype, 128, 1, False, fused=True)
        t.pos = np.array([[len(rows[s]) + who[:r].count(s) for r, s in enumerate(who)]], np.int32)
        pa.pa_norm_rope_append8(pool, *t.args(wq, wk, slots))
        k, v = t.want(t.k, wk)[0], to64(t.v)
        for r, s in enumerate(who):
            rows[s] = rows[s] + [(k[r], v[r])]
        seqs = sorted(rows)
        W = max(len(alloc.table(s)) for s in seqs)
        tables = np.full((len(seqs), W), -1, np.int32)
        for i, s in enumerate(seqs):
            tables[i, :len(alloc.table(s))] = alloc.table(s)
        lens = np.array([alloc.seq_len(s) for s in seqs], np.int32)
        q = torch.from_numpy(rng.standard_normal((len(seqs), Hq, D)).astype(np.float32)).to(dtype).cuda()
        out = torch.empty(len(seqs), Hq, D, device="cuda")
        pa.pa_decode8(pool, q, cuda(tables), cuda(lens), D ** -0.5, out)
        ok8(pa, pool)
        kc, vc, ek, ev = raw(pool)
        kv, vv = values8(kc, ek, kind), values8(vc, ev, kind)
        for i, s in enumerate(seqs):
            L = lens[i]
            assert L == len(rows[s])
            kr, vr = cache_rows(kv, tables[i], L), cache_rows(vv, tables[i], L)
            # decode over what the cache holds: the tolerance of the decode's own tests
            want = attend64(to64(q[i]), kr, vr, D ** -0.5)[0]
            size = np.abs(vr).max()
            a = np.einsum("hgd,htd->hgt", np.abs(to64(q[i])).reshape(Hkv, -1, D), np.abs(kr)).max() * D ** -0.5
            assert np.abs(to64(out[i]) - want).max() <= 2 * (2.0 ** -19 + 2 * a * 2.0 ** -20) * size
            # and the cache holds the rows: the last rounding is off by half a step, what earlier moves of the
            # scale left by less than that together (each was half as large as the next one).  int8: a
            # step is at most 2 / 127 of the largest magnitude; e4m3: 2^-3 of a value, or (subnormal
            # codes) 2^-9 of a scale that is at most 1 / 224 of the largest magnitude
            for x, held in ((np.stack([r[0] for r in rows[s]], 1), kr), (np.stack([r[1] for r in rows[s]], 1), vr)):
                for j in range(0, L, BS):
                    top = np.abs(x[:, j:j + BS]).max((1, 2), keepdims=True)
                    step_ = 2 / 127 * top if kind == "int8" else np.maximum(2.0 ** -3 * np.abs(x[:, j:j + BS]), 2.0 ** -16 * top)
                    assert (np.abs(held[:, j:j + BS] - x[:, j:j + BS]) <= step_ + 2.0 ** -17 * top).all()

    for s in range(3):
        alloc.seq_add(s)
        rows[s] = []
    step({0: 37, 1: 5, 2: 16})
    step({0: 20, 1: 64})
    for _ in range(9):
        step({0: 1, 1: 1, 2: 1})
    alloc.fork(0, 7)
    rows[7] = list(rows[0])
    for _ in range(4):
        step({0: 1, 7: 1, 2: 1})
    step({7: 3, 1: 2})
    alloc.seq_free(1)
    del rows[1]
    step({0: 1, 2: 1, 7: 1})


@pytest.mark.parametrize("kind", KINDS)
def test_a_request_parked_and_brought_back(pa, kind):
    """16-bit decode over the pages that came back equals the 8-bit decode over the parked ones, to the
    tolerance of both (the 16-bit pool holds the parked values exactly in bf16)."""
    rng = np.random.default_rng(2)
    L, Hq, Hkv, dtype = 700, 8, 2, torch.bfloat16
    nb = -(-L // BS)
    pool = filled_pool(pa, rng, 2 * nb, Hkv, dtype)
    pool8 = pa.Pool8(nb, Hkv, type8(kind))
    perm = rng.permutation(2 * nb).astype(np.int32)
    rows = np.full(nb, BS, np.int32)
    rows[-1] = L - BS * (nb - 1)
    park = rng.permutation(nb).astype(np.int32)
    pa.pa_quantize_blocks(pool, cuda(perm[:nb]), pool8, cuda(park), rows=cuda(rows))
    pa.pa_dequantize_blocks(pool8, cuda(park), pool, cuda(perm[nb:]))
    q = torch.from_numpy(rng.standard_normal((1, Hq, D)).astype(np.float32)).to(dtype).cuda()
    lens = cuda(np.array([L], np.int32))
    a, b = torch.empty(1, Hq, D, device="cuda"), torch.empty(1, Hq, D, device="cuda")
    pa.pa_decode8(pool8, q, cuda(park[None]), lens, D ** -0.5, a)
    pa.pa_decode_split(pool, q, cuda(perm[None, nb:]), lens, D ** -0.5, b)
    ok8(pa, pool8)
    ok(pa, pool)
    # 16-bit decode in bf16: weights carried to 2^-17, so 2^-16 of the largest value with the sums
    size = float(pool.v.abs().max())
    assert (a - b).abs().max() <= (2.0 ** -15) * size
