"""Decode over the 8-bit cache against the 64-bit definition.

Tolerance, from the arithmetic (fp32 output): codes, and q scaled by a power of
two, are exact in fp16.  A score is a sum of 128 products in two chains of four
matrix products (16 terms each, accumulated in fp32, cut off rather than rounded:
2^-23 of the partial sums a step at most), one addition and three roundings of
2^-24 (with scale * log2(e)): off by less than 2^-20 of A = scale * sum |q k|.  A
weight is off by that as an exponent, 2^-22 of the exponential and of its two
halves each, the sums by 2^-22 and the join by 2^-21: all weights within 2^-19 + 2
A 2^-20 of themselves, numerator and denominator, so an output is within twice
that of the largest |v| attended.  A 16-bit output adds half of its step."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, attend64, cache_rows, cuda, half_step, rand16, tables_for, to64
from ._ops8 import KINDS, fill8, filled_pool8, ok8, values8

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


class Case:
    def __init__(self, pa, lens, Hq, Hkv, kind, dtype=torch.bfloat16, seed=0, spread=2, width=None):
        self.pa, self.lens, self.Hq, self.Hkv, self.kind, self.dtype = pa, list(lens), Hq, Hkv, kind, dtype
        self.rng = np.random.default_rng(seed + sum(lens) + 7 * Hq)
        self.tables, self.free, n = tables_for(lens, self.rng, width=width)
        self.pool, (self.k, self.v, self.ek, self.ev) = filled_pool8(pa, self.rng, kind, n, Hkv, spread)
        self.q = rand16(self.rng, dtype, len(lens), Hq, D).cuda()

    def refill(self):
        fill8(self.pool, self.k, self.v, self.ek, self.ev)

    def call(self, out_dtype=torch.float32, scale=SCALE, **kw):
        out = torch.full((len(self.lens), self.Hq, D), float("nan"), dtype=out_dtype, device="cuda")
        self.pa.pa_decode8(self.pool, self.q, cuda(self.tables), cuda(np.asarray(self.lens, np.int32)), scale, out, **kw)
        return out

    def reference(self, scale=SCALE):
        """out [B][Hq][128] and its bound, per row."""
        k, v = values8(self.k, self.ek, self.kind), values8(self.v, self.ev, self.kind)
        q = to64(self.q)
        out, bound = np.zeros(q.shape), np.zeros(q.shape[:2] + (1,))
        G = self.Hq // self.Hkv
        for i, L in enumerate(self.lens):
            kr, vr = cache_rows(k, self.tables[i], L), cache_rows(v, self.tables[i], L)
            out[i] = attend64(q[i], kr, vr, scale)[0]
            if L:
                a = np.einsum("hgd,htd->hgt", np.abs(q[i]).reshape(self.Hkv, G, D), np.abs(kr)).max(2) * abs(scale)
                rel = 2 * (2.0 ** -19 + 2 * a * 2.0 ** -20)
                bound[i] = (rel * np.abs(vr).max((1, 2))[:, None]).reshape(-1, 1)
        return out, bound

    def check(self, out, ref=None):
        want, bound = ref or self.reference()
        got = to64(out)
        if out.dtype != torch.float32:
            bound = bound + half_step(out.dtype) * (np.abs(want) + bound) + (2.0 ** -25 if out.dtype == torch.float16 else 0)
        bad = ~(np.abs(got - want) <= bound)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0].tolist(), float(np.nanmax(np.abs(got - want))))


LENS = [
    [1], [16], [17], [0, 5, 0], [33, 1, 15, 16, 0, 17, 100], [700, 3, 250, 90], [5000], [2, 9000, 31, 0, 640],
]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (6, 2), (8, 2), (7, 1), (16, 2), (40, 40)])
def test_against_the_definition(pa, lens, kind, Hq, Hkv):
    c = Case(pa, lens, Hq, Hkv, kind, torch.bfloat16 if Hq % 2 else torch.float16)
    ref = c.reference()
    for out_dtype in (torch.float32, torch.bfloat16, torch.float16):
        c.check(c.call(out_dtype), ref)
    ok8(pa, c.pool)


@pytest.mark.parametrize("G", range(1, 9))
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_groups(pa, G, dtype):
    c = Case(pa, [260, 31, 1111], 3 * G, 3, "e4m3" if G % 2 else "int8", dtype, seed=G)
    c.check(c.call())


@pytest.mark.parametrize("B", [1, 31, 33, 200, 4096])
def test_batches(pa, B):
    rng = np.random.default_rng(B)
    c = Case(pa, rng.integers(0, 60, B).tolist(), 8, 2, "int8", seed=B)
    c.check(c.call(torch.bfloat16))
    ok8(pa, c.pool)


@pytest.mark.parametrize("Hq,Hkv,B", [(6, 1, 3), (4, 2, 9), (8, 4, 15), (8, 4, 16), (12, 2, 40), (4, 2, 80)])
@pytest.mark.parametrize("width", [31, 32, 33, 95, 96, 97, 5000])
def test_tables_of_every_width(pa, Hq, Hkv, B, width):
    """The table's width and the number of segments choose the plan, not the result: both sides of each limit
    (32 and 96 blocks, 64 segments, the SMs), also with lengths far below the width."""
    rng = np.random.default_rng(width * B)
    top = min(width, 97) * BS
    lens = rng.integers(0, top + 1, B)
    lens[:3] = top, 0, top - 15
    c = Case(pa, lens.tolist(), Hq, Hkv, "e4m3" if B % 2 else "int8", seed=B, width=width)
    c.check(c.call())
    ok8(pa, c.pool)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (6, 1)])
@pytest.mark.parametrize("lens", [[3000, 77, 500], [20] * 40, [9000]])
def test_any_blocks_out_of_range(pa, Hq, Hkv, lens):
    """A third of the table's entries name no block, first and last ones among them: softmax over what is left."""
    c = Case(pa, lens, Hq, Hkv, "int8", seed=4)
    k, v = values8(c.k, c.ek, c.kind), values8(c.v, c.ev, c.kind)
    q, want, bound = to64(c.q), np.zeros((len(lens), Hq, D)), 0.0
    for i, L in enumerate(lens):
        keep = np.ones(L, bool)
        kr, vr = cache_rows(k, c.tables[i], L), cache_rows(v, c.tables[i], L)
        for j in range(-(-L // BS)):
            if c.rng.random() < 0.3 or (i == 0 and j in (0, (L - 1) // BS)):
                c.tables[i, j] = int(c.rng.choice([-1, -(1 << 31), c.pool.num_blocks, (1 << 31) - 1]))
                keep[j * BS:(j + 1) * BS] = False
        want[i] = attend64(q[i], kr[:, keep], vr[:, keep], SCALE)[0]
        a = np.einsum("hgd,htd->hgt", np.abs(q[i]).reshape(Hkv, -1, D), np.abs(kr)).max() * SCALE
        bound = max(bound, 2 * (2.0 ** -19 + 2 * a * 2.0 ** -20) * np.abs(vr).max())
    assert np.abs(to64(c.call()) - want).max() <= bound
    assert pa.pa_check8(c.pool)[0] == pa.PA_ERR_DEVICE_CHECK


@pytest.mark.parametrize("kind", KINDS)
def test_what_is_behind_the_end_does_not_count(pa, kind):
    """NaN codes, NaN exponents and table entries that name no block, behind the sequences' ends."""
    c = Case(pa, [5, 16, 47, 0], 8, 2, kind, width=6)
    want = c.call()
    k, v, ek, ev = (x.copy() for x in (c.k, c.v, c.ek, c.ev))
    used = set()
    for i, L in enumerate(c.lens):
        used |= set(c.tables[i, :-(-L // BS)].tolist())
        if L % BS:
            b = c.tables[i, L // BS]
            k[b, :, L % BS:] = v[b, :, L % BS:] = 0x7F if kind == "e4m3" else 0x80
    for b in set(range(len(ek))) - used:
        ek[b] = ev[b] = 255
    fill8(c.pool, k, v, ek, ev)
    c.tables[c.tables < 0] = 1 << 30
    assert torch.equal(c.call(), want)
    ok8(pa, c.pool)


def test_blocks_out_of_range_count_as_not_attended(pa):
    c = Case(pa, [70, 40, 20], 8, 2, "e4m3")
    bad = int(c.pool.num_blocks)
    c.tables[0, 1], c.tables[2, :2] = bad, -5
    got = c.call()
    code, detail = pa.pa_check8(c.pool)
    assert code == pa.PA_ERR_DEVICE_CHECK and detail in (bad, -5)
    assert (got[2] == 0).all(), "nothing to attend"
    c.lens = [70 - BS, 40, 0]
    c.tables[0, 1:4] = c.tables[0, 2:5]
    c.check(got)


def test_lengths_out_of_range_are_clamped(pa):
    c = Case(pa, [40, 48, 10], 8, 2, "int8")
    c.lens = [40, 48, 0]
    want = c.call()
    c.lens = [40, 1000, -3]
    assert torch.equal(c.call(), want)
    code, detail = pa.pa_check8(c.pool)
    assert code == pa.PA_ERR_DEVICE_CHECK and detail in (1000, -3)


@pytest.mark.parametrize("lens", [[60], [30, 6000, 4]])
@pytest.mark.parametrize("kind", KINDS)
def test_scales_that_differ_widely(pa, lens, kind):
    """Values of one block 2^60 above those of the others, with weights near zero and not."""
    c = Case(pa, lens, 8, 2, kind, seed=3)
    c.ev[c.tables[0, 1]] += 60
    c.ev[c.tables[0, 2]] = 1
    i = len(lens) // 2
    c.ek[c.tables[i, 0]] = 0  # 2^-127: scores of zero
    c.refill()
    c.check(c.call())


@pytest.mark.parametrize("e", [0, 1, 40, 247])
@pytest.mark.parametrize("L", [9, 3000])
def test_values_at_the_ends_of_the_exponents(pa, e, L):
    """All of V at one exponent: the outputs scale with it (2^-127 to 2^120; fp32 output, below its largest number)."""
    c = Case(pa, [L], 4, 1, "int8", seed=e)
    c.ev[:] = 127
    c.refill()
    want = c.call().double()
    c.ev[:] = e
    c.refill()
    # (subnormal outputs are rounded to 2^-149)
    got, size = c.call().double(), 2.0 ** (e - 127)
    assert (got - want * size).abs().max() <= 2.0 ** -22 * (want * size).abs().max() + 2.0 ** -148


def test_tokens_that_one_outweighs_keep_their_values(pa):
    """4,096 tokens behind one that outweighs each by 2^26: their sum is 2^-14 of the weight."""
    c = Case(pa, [4097], 4, 1, "int8", torch.float16)
    c.q.fill_(1.0)
    c.k[:], c.ek[:], c.v[:], c.ev[:] = 0, 127, 100, 127
    b = c.tables[0, 0]
    c.k[b, :, 0] = 1
    c.v[b, :, 0] = 0
    c.refill()
    scale = 26 * np.log(2) / D
    got = to64(c.call(scale=scale))
    want = 100 * 4096 / (4096 + 2.0 ** 26)
    assert np.abs(got / want - 1).max() < 2.0 ** -9, "weights of 2^-26 are carried to 2^-35"


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 2.0 ** 20, 2.0 ** 100])
def test_queries_of_any_size(pa, size):
    """The scale of the call takes the size back: the same result as at size 1."""
    c = Case(pa, [300, 20], 8, 2, "e4m3")
    want = c.call()
    c.q *= size
    assert torch.equal(c.call(scale=SCALE / size), want)


def test_small_elements_beside_a_large_one(pa):
    """q with one element 2^20 above the others, its keys zero: the others still count in full."""
    c = Case(pa, [200], 8, 2, "int8")
    c.q[:, :, 5] = 2.0 ** 20
    c.k[:, :, :, 5] = 0
    c.refill()
    c.check(c.call())


NANS = [(kind, where) for kind in KINDS for where in ("key code", "value code", "key scale", "value scale", "query")
        if kind == "e4m3" or "code" not in where]  # (int8 has no NaN code)


@pytest.mark.parametrize("kind,where", NANS)
@pytest.mark.parametrize("t", [0, 37, 4999])
def test_nan_reaches_the_rows_that_attend_it(pa, kind, where, t):
    c = Case(pa, [20, 5000, 64], 8, 2, kind)
    clean = c.call()
    b, r = c.tables[1, t // BS], t % BS
    rows = slice(4, 8)  # of kv head 1
    if where == "key code":
        c.k[b, 1, r, 9] = 0xFF
    elif where == "value code":
        c.v[b, 1, r, 9] = 0x7F
    elif where == "key scale":
        c.ek[b, 1] = 255
    elif where == "value scale":
        c.ev[b, 1] = 255
    else:
        c.q[1, 6, 3] = float("nan")
        rows = slice(6, 7)
    c.refill()
    got = c.call()
    hit = got[1, rows, 9:10] if where == "value code" else got[1, rows]
    assert torch.isnan(hit).all()
    if where == "value code":
        got[1, rows, 9] = clean[1, rows, 9]
    else:
        got[1, rows] = clean[1, rows]
    assert torch.equal(got, clean)


def test_infinite_queries_give_nan_and_leave_the_others(pa):
    c = Case(pa, [50, 50], 8, 2, "e4m3")
    clean = c.call()
    c.q[0, 2, 4] = float("inf")
    got = c.call()
    assert torch.isnan(got[0, 2]).all()
    got[0, 2] = clean[0, 2]
    assert torch.equal(got, clean)


def test_the_result_does_not_depend_on_place_workspace_stream_or_graph(pa):
    c = Case(pa, [900, 3, 4000, 77], 12, 2, "e4m3", torch.float16, seed=5)
    want = c.call()
    lens, tables = cuda(np.asarray(c.lens, np.int32)), cuda(c.tables)
    ws = pa.decode8_workspace_for(c.pool, c.q, tables)
    ws.fill_(0xFF)
    assert torch.equal(c.call(workspace=ws), want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    pa.pa_decode8(c.pool, c.q, tables, lens, SCALE, out, stream=st)
    st.synchronize()
    assert torch.equal(out, want)
    # two captured calls that share a workspace, replayed in turn
    other, q2 = torch.empty_like(want), -c.q
    graphs = []
    for q, o in ((c.q, out), (q2, other)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_decode8(c.pool, q, tables, lens, SCALE, o, workspace=ws)
        graphs.append(g)
    out.zero_()
    for g in graphs * 3:
        g.replay()
    assert torch.equal(out, want)
    c.q = q2
    assert torch.equal(c.call(), other)
    # another placement of the same blocks
    c.q = -q2
    perm = c.rng.permutation(c.pool.num_blocks)
    for x in (c.k, c.v, c.ek, c.ev):
        x[perm] = x.copy()
    c.tables = np.where(c.tables >= 0, perm[np.maximum(c.tables, 0)], -1).astype(np.int32)
    c.refill()
    assert torch.equal(c.call(), want)


def test_writes_stay_inside(pa):
    """Guards around out and the workspace of the documented size."""
    c = Case(pa, [16 * n for n in range(1, 40)] + [3000], 8, 2, "int8")
    B = len(c.lens)
    tables, lens = cuda(c.tables), cuda(np.asarray(c.lens, np.int32))
    n = pa.lib.pa_decode8_workspace_bytes(c.pool.handle8, B, 8, tables.shape[1])
    ws = torch.full((n + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    out = torch.full((B + 2, 8, D), 7.0, device="cuda")
    pa.pa_decode8(c.pool, c.q, tables, lens, SCALE, out[1:-1], workspace=ws[256:256 + n])
    assert (ws[:256] == 0xAB).all() and (ws[256 + n:] == 0xAB).all()
    assert (out[0] == 7).all() and (out[-1] == 7).all()
    c.check(out[1:-1])


def test_blocks_behind_four_gigabytes(pa):
    """The top blocks of a 4.9 GB pool give the bits of a small one."""
    rng = np.random.default_rng(21)
    small, (k, v, ek, ev) = filled_pool8(pa, rng, "e4m3", 60, 8)
    tables = rng.permutation(60).reshape(2, 30).astype(np.int32)
    lens = cuda(np.array([470, 333], np.int32))
    q = rand16(rng, torch.bfloat16, 2, 32, D).cuda()
    want, got = (torch.empty(2, 32, D, device="cuda") for _ in range(2))
    pa.pa_decode8(small, q, cuda(tables), lens, SCALE, want)
    big = 150000
    pool = pa.Pool8(big, 8, torch.float8_e4m3fn)
    for t, x in ((pool.k, k), (pool.v, v)):
        t[big - 60:].copy_(torch.from_numpy(x).cuda().view(torch.float8_e4m3fn))
    for t, x in ((pool.k_scale, ek), (pool.v_scale, ev)):
        t[big - 60:].copy_(torch.from_numpy(x).cuda().view(torch.float8_e8m0fnu))
    pa.pa_decode8(pool, q, cuda(tables + big - 60), lens, SCALE, got)
    assert torch.equal(got, want)
    ok8(pa, pool)
    pool.close()


def test_refusals(pa):
    c = Case(pa, [20, 30], 8, 2, "int8")
    t, lens = cuda(c.tables), cuda(np.asarray(c.lens, np.int32))
    out = torch.zeros(2, 8, D, device="cuda")
    for scale in (float("nan"), float("inf")):
        with pytest.raises(pa.PagedAttentionError):
            pa.pa_decode8(c.pool, c.q, t, lens, scale, out)
    ws = pa.decode8_workspace_for(c.pool, c.q, t)
    for bad in (ws[:-1], torch.empty(ws.numel() + 16, dtype=torch.uint8, device="cuda")[16:]):
        with pytest.raises(pa.PagedAttentionError):
            pa.pa_decode8(c.pool, c.q, t, lens, SCALE, out, workspace=bad)
    with pytest.raises(pa.PagedAttentionError):  # 9 query heads a kv head
        pa.pa_decode8(c.pool, rand16(c.rng, torch.bfloat16, 2, 18, D).cuda(), t, lens, SCALE, torch.zeros(2, 18, D, device="cuda"),
                      workspace=ws)
    with pytest.raises(ValueError):
        pa.pa_decode8(c.pool, c.q, t[:1], lens, SCALE, out)
    with pytest.raises(ValueError):
        pa.pa_decode8(c.pool, c.q, t, lens, SCALE, out[:, :4].contiguous())
    with pytest.raises(ValueError):
        pa.pa_decode8(c.pool, c.q, t, lens, SCALE, out.double())
    L, none = pa.lib, None
    args = (c.q.data_ptr(), pa.PA_BF16, t.data_ptr(), t.shape[1], lens.data_ptr())
    tail = (out.data_ptr(), pa.PA_FP32, ws.data_ptr(), ws.numel(), none)
    assert L.pa_decode8(c.pool.handle8, *args, 4097, 8, 0.1, *tail) == pa.PA_ERR_UNSUPPORTED
    assert L.pa_decode8(c.pool.handle8, *args, 2, 7, 0.1, *tail) == pa.PA_ERR_INVALID
    assert L.pa_decode8(c.pool.handle8, args[0], pa.PA_FP32, *args[2:], 2, 8, 0.1, *tail) == pa.PA_ERR_INVALID
    assert L.pa_decode8(c.pool.handle8, *args[:3], 1 << 27, args[4], 2, 8, 0.1, *tail) == pa.PA_ERR_UNSUPPORTED
    assert L.pa_decode8_workspace_bytes(c.pool.handle8, 4097, 8, 1) == 0
    assert (out == 0).all()


def test_pools_of_the_other_kind_are_refused(pa):
    p16, p8 = pa.Pool(2, 2, torch.bfloat16), pa.Pool8(2, 2, torch.int8)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q, out = (torch.zeros(1, 4, D, dtype=torch.bfloat16, device="cuda") for _ in "qo")
    rows, slots = torch.zeros(1, 2, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    for call in (lambda: pa.pa_decode8(p16, q, i32(0)[None], i32(1), SCALE, out), lambda: pa.pa_cache_append8(p16, rows, rows, slots),
                 lambda: pa.pa_copy_blocks8(p16, i32(0), i32(1)), lambda: pa.pa_check8(p16)):
        with pytest.raises(TypeError, match="takes a Pool8"):
            call()
    q8, rows8 = q.to(torch.int8), rows.to(torch.int8)
    for call in (lambda: pa.pa_decode(p8, q8, i32(0)[None], i32(1), SCALE, out), lambda: pa.pa_copy_blocks(p8, i32(0), i32(1)),
                 lambda: pa.pa_cache_append(p8, rows8, rows8, slots), lambda: pa.pa_check(p8),
                 lambda: pa.pa_decode_split(p8, q8, i32(0)[None], i32(1), SCALE, out)):
        with pytest.raises(TypeError, match="takes a Pool, got a Pool8"):
            call()


def test_the_pool_lives_as_long_as_its_views(pa):
    pool = pa.Pool8(4, 2, torch.int8)
    k, s = pool.k, pool.v_scale
    k.fill_(3)
    del pool
    torch.cuda.synchronize()
    assert (k == 3).all() and (s.view(torch.uint8) == 0).all()
