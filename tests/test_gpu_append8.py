"""The cache write in 8 bits.  Without norms and rotation every step is exact but
the one rounding to a code, so codes and exponents are the definition's, byte for
byte.  With them K rows carry the errors of the 16-bit append (2^-18 of |x| + |y|)
before that rounding: an exponent is the one of a magnitude within that, and a
code is within half of its step and the error."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, cuda, to64
from ._ops8 import KINDS, decode8, encode8, filled_pool8, need8, ok8, rand_rows, raw, runs_of, scale8, type8, write8
from .test_gpu_norm_rope import EPS, Tokens, pair_size, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


def slots_for(rng, n_blocks, pieces, shuffle=False):
    """Slots of sequences' new tokens: (held, new) each, on blocks of their own in random places."""
    perm, at, slots = rng.permutation(n_blocks), 0, []
    for held, new in pieces:
        nb = -(-(held + new) // BS)
        table = perm[at:at + nb]
        at += nb
        p = np.arange(held, held + new)
        slots.append(table[p // BS] * BS + p % BS)
    return slots


def same(pool, want):
    for got, ref, name in zip(raw(pool), want, ("k codes", "v codes", "k exponents", "v exponents")):
        assert np.array_equal(got, ref), (name, np.argwhere(got != ref)[:5].tolist())


def write_and_compare(pa, kind, dtype, hkv, slots, n_blocks, seed, rows=None, spread=2):
    rng = np.random.default_rng(seed)
    pool, (k, v, ek, ev) = filled_pool8(pa, rng, kind, n_blocks, hkv, spread)
    n = len(slots)
    kn, vn = rows or (rand_rows(rng, dtype, n, hkv), rand_rows(rng, dtype, n, hkv))
    slots = np.asarray(slots, np.int64)
    k, ek = write8(k, ek, to64(kn), slots, kind)
    v, ev = write8(v, ev, to64(vn), slots, kind)
    pa.pa_cache_append8(pool, kn, vn, cuda(slots))
    same(pool, (k, v, ek, ev))
    return pool


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hkv", [1, 2, 5, 8])
@pytest.mark.parametrize("pieces", [
    [(0, 1)], [(7, 1)], [(0, 16)], [(3, 40)], [(15, 2)], [(0, 15), (1, 15), (31, 18)],
    [(h, 1) for h in range(0, 70, 2)], [(5, 5)] * 16, [(0, 257)], [(9, 100), (0, 1), (16, 1), (17, 33), (12, 4), (13, 4)],
])
def test_sequences_in_order(pa, kind, dtype, hkv, pieces):
    rng = np.random.default_rng(len(pieces) * 31 + hkv)
    nb = sum(-(-(h + n) // BS) for h, n in pieces) + 2
    slots = np.concatenate(slots_for(rng, nb, pieces))
    ok8(pa, write_and_compare(pa, kind, dtype, hkv, slots, nb, 3))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seed", range(6))
def test_random_batches_with_padding(pa, kind, seed):
    rng = np.random.default_rng(100 + seed)
    pieces = [(int(rng.integers(0, 60)), int(rng.integers(1, 40))) for _ in range(int(rng.integers(1, 30)))]
    nb = sum(-(-(h + n) // BS) for h, n in pieces) + 2
    parts = slots_for(rng, nb, pieces)
    out = []
    for p in parts:  # padding rows between and behind the sequences
        out += [p, np.full(int(rng.integers(0, 20)) * int(rng.integers(0, 2)), -int(rng.integers(1, 9)))]
    ok8(pa, write_and_compare(pa, kind, torch.bfloat16, 3, np.concatenate(out), nb, seed, spread=int(rng.integers(0, 6))))


@pytest.mark.parametrize("kind", KINDS)
def test_rows_of_many_sizes(pa, kind):
    """From the smallest numbers to the largest: exponents at their floor, far apart in one block, zero rows, ties."""
    for dtype, sizes in ((torch.bfloat16, [2.0 ** -133, 2.0 ** -126, 1e-30, 1.0, 1e30, 3e38]),
                         (torch.float16, [6e-8, 1e-4, 1.0, 6e4])):
        rng = np.random.default_rng(9)
        nb, hkv = len(sizes) ** 2 + 1, 2
        rows, slots = [], []
        for a, x in enumerate(sizes):
            for b, y in enumerate(sizes):
                s = a * len(sizes) + b
                rows += [x, y]
                slots += [s * BS, s * BS + 1]
        x = torch.from_numpy(rng.uniform(-1, 1, (len(rows), hkv, D)).astype(np.float32)).cuda()
        x = (x * torch.tensor(rows, device="cuda")[:, None, None]).to(dtype)
        x[3], x[8, 0] = 0.0, torch.arange(D, device="cuda").to(dtype) / 2  # (halves: ties)
        write_and_compare(pa, kind, dtype, hkv, slots, nb, 10, rows=(x, x.flip(0).contiguous()))
        # one token at a time: the same rows, the second one on top of the first
        pool = pa.Pool8(nb, hkv, type8(kind))
        k, v, ek, ev = raw(pool)
        for r in (0, 1):
            at = np.asarray(slots[r::2], np.int64)
            kn, vn = x[r::2].contiguous(), x.flip(0)[r::2].contiguous()
            pa.pa_cache_append8(pool, kn, vn, cuda(at))
            k, ek = write8(k, ek, to64(kn), at, kind)
            v, ev = write8(v, ev, to64(vn), at, kind)
        same(pool, (k, v, ek, ev))


@pytest.mark.parametrize("kind", KINDS)
def test_rows_that_are_not_finite_mark_their_tile(pa, kind):
    rng = np.random.default_rng(11)
    pool, (k, v, ek, ev) = filled_pool8(pa, rng, kind, 4, 2)
    kn, vn = rand_rows(rng, torch.bfloat16, 20, 2), rand_rows(rng, torch.bfloat16, 20, 2)
    kn[3, 1, 60], vn[18, 0, 5] = float("nan"), float("-inf")
    slots = np.concatenate([np.arange(4, 16), np.arange(32, 40)]).astype(np.int64)
    pa.pa_cache_append8(pool, kn, vn, cuda(slots))
    k1, ek1 = write8(k, ek, to64(kn), slots, kind)
    v1, ev1 = write8(v, ev, to64(vn), slots, kind)
    gk, gv, gek, gev = raw(pool)
    assert np.array_equal(gek, ek1) and np.array_equal(gev, ev1)
    assert gek[0, 1] == 255 and gev[2, 0] == 255 and (gek == 255).sum() == 1 and (gev == 255).sum() == 1
    for got, ref, e in ((gk, k1, gek), (gv, v1, gev)):
        assert np.array_equal(got[e != 255], ref[e != 255])
    # it stays so until the block is started afresh
    pa.pa_cache_append8(pool, *(rand_rows(rng, torch.bfloat16, 1, 2) for _ in "kv"), cuda(np.array([5], np.int64)))
    assert raw(pool)[2][0, 1] == 255
    pa.pa_cache_append8(pool, *(rand_rows(rng, torch.bfloat16, 2, 2) for _ in "kv"), cuda(np.array([0, 1], np.int64)))
    assert raw(pool)[2][0, 1] != 255
    ok8(pa, pool)


def test_slots_out_of_range_are_skipped_and_reported(pa):
    rng = np.random.default_rng(12)
    for bad in (48, 1 << 40):
        slots = np.array([44, 45, 46, 47, bad, bad + 1, 3, 4], np.int64)
        pool = write_and_compare(pa, "int8", torch.float16, 2, slots, 3, 13)
        assert pa.pa_check8(pool) == (pa.PA_ERR_DEVICE_CHECK, bad)
        ok8(pa, pool)


CASES = [  # pieces, Hq, Hkv, dtype, kind, rot, axes, interleaved, fused, norms
    ([(600 + 3 * i, 1) for i in range(20)], 32, 8, torch.bfloat16, "e4m3", 128, 1, False, True, "qk"),
    ([(0, 100), (5, 41), (16, 1)], 12, 2, torch.float16, "int8", 64, 2, True, False, "qk"),
    ([(3, 4)] * 9, 8, 8, torch.bfloat16, "int8", 96, 1, False, True, "k"),
    ([(0, 33), (31, 2)], 5, 5, torch.float16, "e4m3", 16, 3, False, False, "q"),
    ([(8, 700)], 10, 2, torch.bfloat16, "e4m3", 128, 1, True, True, ""),
    # query rows that wait in shared memory
    ([(8, 300), (0, 290), (77, 220)], 30, 3, torch.float16, "int8", 64, 1, True, False, "qk"),
    ([(5, 400), (300, 380)], 32, 2, torch.bfloat16, "e4m3", 128, 1, False, True, "q"),
    ([(1, 900)], 28, 1, torch.float16, "e4m3", 96, 1, False, True, "k"),
]


@pytest.mark.parametrize("pieces,Hq,Hkv,dtype,kind,rot,n_axes,interleaved,fused,norms", CASES)
def test_norms_and_rotation_on_the_way(pa, pieces, Hq, Hkv, dtype, kind, rot, n_axes, interleaved, fused, norms):
    rng = np.random.default_rng(len(pieces) + rot)
    nb = sum(-(-(h + n) // BS) for h, n in pieces) + 2
    slots = np.concatenate(slots_for(rng, nb, pieces) + [np.full(3, -1)])
    n = len(slots)
    t = Tokens(rng, n, Hq, Hkv, dtype, rot, n_axes, interleaved, fused)
    wq, wk = (weight(rng, dtype) if x in norms else None for x in "qk")
    pool, (k0, v0, ek0, ev0) = filled_pool8(pa, rng, kind, nb, Hkv)
    pa.pa_norm_rope_append8(pool, *t.args(wq, wk, slots), eps=EPS, interleaved=interleaved)
    ok8(pa, pool)
    # the query rows are the 16-bit append's, bit for bit; so are the value codes those without norms
    p16 = pa.Pool(nb, Hkv, dtype)
    q8 = t.q_out.clone()
    pa.pa_norm_rope_append(p16, *t.args(wq, wk, slots), eps=EPS, interleaved=interleaved)
    assert torch.equal(q8, t.q_out)
    k, v, ek, ev = raw(pool)
    v1, ev1 = write8(v0, ev0, to64(t.v), slots, kind)
    assert np.array_equal(v, v1) and np.array_equal(ev, ev1)
    ref, normed = t.want(t.k, wk)
    err = 2.0 ** -18 * pair_size(normed, rot, interleaved)
    done = np.zeros((nb, BS), bool)
    for run in runs_of(slots, nb * BS):
        b, off = int(slots[run[0]]) // BS, int(slots[run[0]]) % BS
        at = off + np.arange(len(run))
        done[b, at] = True
        other = np.setdiff1d(np.arange(BS), at)
        for h in range(Hkv):
            x, slack = ref[run, h], err[run, h]
            floor = int(ek0[b, h]) if off else 0
            e = int(ek[b, h])
            assert e in {max(floor, need8(a, kind)) for a in (max((np.abs(x) - slack).max(), 0), (np.abs(x) + slack).max())}
            s = float(scale8(e))
            # half a step of the code at |x| (and at the top half a step of the last one)
            step = np.full_like(x, s) if kind == "int8" else s * 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x) / s, 2.0 ** -6))) - 3)
            assert (np.abs(decode8(k[b, h, at], kind) * s - x) <= step / 2 * (1 + 2.0 ** -10) + slack).all()
            held = k0[b, h, other]
            if off and e > ek0[b, h]:
                held = encode8(decode8(held, kind) * 2.0 ** (int(ek0[b, h]) - e), kind)
            assert np.array_equal(k[b, h, other], held)
    untouched = ~done.any(1)
    assert np.array_equal(k[untouched], k0[untouched]) and np.array_equal(ek[untouched], ek0[untouched])


def test_streams_graphs_and_repeats(pa):
    """A captured write replayed on a pool in the same state gives the same bytes; writing the same rows again changes nothing."""
    rng = np.random.default_rng(14)
    pieces = [(9, 20), (0, 3), (30, 1)]
    slots = np.concatenate(slots_for(rng, 9, pieces))
    t = Tokens(rng, len(slots), 8, 2, torch.bfloat16, 128, 1, False)
    w = weight(rng, torch.bfloat16)
    pool, state = filled_pool8(pa, rng, "e4m3", 9, 2)
    args = t.args(w, w, slots)
    pa.pa_norm_rope_append8(pool, *args)
    want = raw(pool)
    pa.pa_norm_rope_append8(pool, *args)
    same(pool, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_norm_rope_append8(pool, *args)
    from ._ops8 import fill8
    fill8(pool, *state)
    graph.replay()
    same(pool, want)
    fill8(pool, *state)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    pa.pa_norm_rope_append8(pool, *args, stream=st)
    st.synchronize()
    same(pool, want)


def test_rows_behind_four_gigabytes(pa):
    """The top blocks of a 4.9 GB pool get the bytes that a small pool gets."""
    rng = np.random.default_rng(15)
    big, hkv, n = 150000, 8, 90
    small = pa.Pool8(8, hkv, torch.int8)
    kn, vn = rand_rows(rng, torch.float16, n, hkv), rand_rows(rng, torch.float16, n, hkv)
    slots = np.arange(20, 20 + n).astype(np.int64)
    pa.pa_cache_append8(small, kn, vn, cuda(slots))
    pool = pa.Pool8(big, hkv, torch.int8)
    pa.pa_cache_append8(pool, kn, vn, cuda(slots + (big - 8) * BS))
    for a, b in ((pool.k, small.k), (pool.v, small.v), (pool.k_scale, small.k_scale), (pool.v_scale, small.v_scale)):
        assert np.array_equal(a[big - 8:].view(torch.uint8).cpu().numpy(), b.view(torch.uint8).cpu().numpy())
    ok8(pa, pool)
    pool.close()


def test_refusals(pa):
    rng = np.random.default_rng(16)
    pool = pa.Pool8(2, 2, torch.int8)
    k = rand_rows(rng, torch.float16, 3, 2)
    s = cuda(np.arange(3).astype(np.int64))
    with pytest.raises(TypeError):
        pa.pa_cache_append8(pool, k, k.bfloat16(), s)
    with pytest.raises(ValueError):
        pa.pa_cache_append8(pool, k, k[:2], s)
    with pytest.raises(ValueError, match="contiguous"):
        pa.pa_cache_append8(pool, k.transpose(0, 1).contiguous().transpose(0, 1), k, s)
    with pytest.raises(TypeError):
        pa.pa_cache_append8(pool, k, k, s.int())
    t = Tokens(rng, 3, 4, 2, torch.float16, 128, 1, False)
    with pytest.raises(TypeError):
        pa.pa_norm_rope_append8(pool, *t.args(weight(rng, torch.bfloat16), None, range(3)))
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_norm_rope_append8(pool, *t.args(None, None, range(3)), eps=-1.0)
    pa.pa_cache_append8(pool, k[:0], k[:0], s[:0])
    assert not pool.k.view(torch.uint8).any()
