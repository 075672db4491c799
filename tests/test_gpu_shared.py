"""Shared-prefix decode for groups of any size, against the 64-bit definition
of attention (the operator is an exact rearrangement of it).

Tolerance with fp32 output, from the arithmetic: a score is off by at most 128 *
2^-23 of sum |k q| * scale =: A (natural-log units; the tensor core may truncate
each addition) and 2^-22 of itself, so each weight by e = 128 * 2^-23 A +
2^-21 (1 + A) relative, twice (weight and sum); the value product carries the
weights to 2^-17 and adds in fp32 (L * 2^-23, truncating).  The output is a
weighted mean of values: off by at most (2 e + 2^-17 + L 2^-23 + 2^-20) * max
|v|.  A 16-bit output adds the weights' own rounding (half a step of the pool's
type) and the output's."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, attend64, cache_rows, cuda, filled_pool, half_step, ok, rand16, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


class Shared:
    """A batch whose sequences share prefixes: groups of (members, prefix
    blocks, own tokens of each member); alone: own tokens of the others."""

    def __init__(self, pa, groups, alone, Hq, Hkv, dtype, seed=0, order="mixed", spare_width=1):
        rng = np.random.default_rng(seed)
        self.pa, self.Hq, self.Hkv, self.dtype = pa, Hq, Hkv, dtype
        seqs = []  # (group or -1, prefix blocks, own tokens)
        for k, (P, own) in enumerate(groups):
            seqs += [(k, P, t) for t in own]
        seqs += [(-1, 0, t) for t in alone]
        at = rng.permutation(len(seqs)) if order == "mixed" else np.arange(len(seqs))
        seqs = [seqs[x] for x in at]
        B = len(seqs)
        self.lens = np.array([P * BS + t for _, P, t in seqs], np.int32)
        W = max(1, max(-(-int(L) // BS) for L in self.lens)) + spare_width
        n = sum(P for P, _ in groups) + sum(-(-t // BS) for _, _, t in seqs) + 5
        free = list(rng.permutation(n))
        pre = [[free.pop() for _ in range(P)] for P, _ in groups]
        self.tables = np.full((B, W), -1, np.int32)
        for i, (k, P, t) in enumerate(seqs):
            if k >= 0:
                self.tables[i, :P] = pre[k]
            own = -(-t // BS)
            self.tables[i, P:P + own] = [free.pop() for _ in range(own)]
        self.members = np.concatenate([np.nonzero([s[0] == k for s in seqs])[0] for k in range(len(groups))] or
                                      [np.zeros(0)]).astype(np.int32)
        self.start = np.cumsum([0] + [len(o) for _, o in groups]).astype(np.int32)
        self.prefix = np.array([P for P, _ in groups], np.int32)
        self.pool = filled_pool(pa, rng, n, Hkv, dtype)
        self.q = rand16(rng, dtype, B, Hq, D).cuda()
        self.B, self.n = B, n

    def call(self, out_dtype=torch.float32, scale=D ** -0.5, **change):
        out = torch.full((self.B, self.Hq, D), float("nan"), dtype=out_dtype, device="cuda")
        a = dict(block_tables=cuda(self.tables), seq_lens=cuda(self.lens), group_start=cuda(self.start),
                 members=cuda(self.members), prefix_blocks=cuda(self.prefix))
        a.update(change)
        self.pa.pa_decode_shared(self.pool, self.q, scale=scale, out=out, **a)
        return out

    def check(self, out, scale=D ** -0.5, rows=None):
        k64, v64, q64, got = to64(self.pool.k), to64(self.pool.v), to64(self.q), to64(out)
        assert np.isfinite(got).all()
        G = self.Hq // self.Hkv
        for i in (range(self.B) if rows is None else rows):
            L = int(self.lens[i])
            k, v = cache_rows(k64, self.tables[i], L), cache_rows(v64, self.tables[i], L)
            ref, _ = attend64(q64[i], k, v, scale)
            if L == 0:
                assert (got[i] == 0).all()
                continue
            a = float(np.einsum("hgd,htd->hgt", np.abs(q64[i]).reshape(self.Hkv, G, D), np.abs(k)).max()) * abs(scale)
            e = 128 * 2.0 ** -23 * a + 2.0 ** -21 * (1 + a)
            tol = 2 * e + 2.0 ** -17 + L * 2.0 ** -23 + 2.0 ** -20
            bound = tol * np.abs(v).max()
            if out.dtype != torch.float32:
                bound = bound + half_step(self.dtype) * np.abs(v).max()
                bound = bound + half_step(out.dtype) * (np.abs(ref) + bound) + 2.0 ** -25
            err = np.abs(got[i] - ref)
            assert (err <= bound).all(), (i, L, float(err.max()), float(np.max(bound)))


CASES = [  # groups, alone, Hq, Hkv, dtype
    ([(1, [0, 1])], [], 4, 1, torch.bfloat16),
    ([(1, [5])], [0, 1, 40], 8, 8, torch.float16),                 # a group of one; rows 1
    ([(8, [1, 2, 3, 4])], [], 12, 2, torch.float16),               # one whole chunk
    ([(9, [16, 17, 0, 33])], [7], 16, 2, torch.bfloat16),          # a chunk and a block
    ([(16, [10] * 32)], [], 4, 1, torch.bfloat16),                 # 128 rows: one tile
    ([(17, [10] * 33)], [], 4, 1, torch.bfloat16),                 # 132 rows: two tiles
    ([(5, [3] * 64)], [], 4, 1, torch.float16),                    # 256 rows
    ([(5, [3] * 65)], [2], 4, 1, torch.float16),                   # 260 rows: two items
    ([(40, [100, 1, 0] * 6), (3, [7, 8]), (0, [9, 40])], [0, 300], 32, 8, torch.bfloat16),
    ([(100, [20] * 5), (130, [60] * 9)], [1000], 40, 40, torch.float16),
    ([(300, [31] * 70)], [], 21, 3, torch.bfloat16),               # G = 7, 490 rows
    ([(700, [5] * 3)], [], 6, 1, torch.float16),
    ([(2, [1, 2])] * 45, [], 5, 1, torch.bfloat16),                # more groups than a warp
]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_definition(pa, case, out_dtype):
    c = Shared(pa, *CASES[case], seed=case)
    out = c.call(out_dtype)
    ok(pa, c.pool)
    c.check(out)
    c.pool.close()


def test_no_groups_is_the_plain_decode(pa):
    c = Shared(pa, [], [10, 700, 0, 33], 8, 2, torch.bfloat16)
    out = c.call()
    ok(pa, c.pool)
    c.check(out)
    c.pool.close()


def test_groups_found_from_the_tables(pa):
    c = Shared(pa, [(40, [100, 1, 0] * 6), (3, [7, 8])], [0, 300], 32, 8, torch.bfloat16)
    gs, mem, pre = pa.cascade_groups(c.tables, c.lens, 32, 8, max_members=c.B)
    assert sorted(pre.tolist()) == [3, 40] and sorted(np.diff(gs).tolist()) == [2, 18]
    out = c.call(group_start=cuda(gs), members=cuda(mem), prefix_blocks=cuda(pre))
    ok(pa, c.pool)
    c.check(out)
    c.pool.close()


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
def test_scales(pa, scale):
    """Zero (means), negative, and scores of hundreds (the maximum moves often)."""
    c = Shared(pa, [(33, [20] * 40)], [], 8, 2, torch.float16, seed=3)
    out = c.call(scale=scale)
    ok(pa, c.pool)
    c.check(out, scale=scale)
    c.pool.close()


def test_rising_scores_move_the_maximum(pa):
    """Keys grow along the prefix, so every chunk's maximum passes the last."""
    c = Shared(pa, [(64, [20] * 34)], [], 8, 2, torch.float16, seed=4)
    first = c.tables[c.members[0]]
    for j in range(64):
        c.pool.k[int(first[j])] *= 0.05 * j
    out = c.call()
    ok(pa, c.pool)
    c.check(out)
    c.pool.close()


def test_unused_slots_hold_nan(pa):
    c = Shared(pa, [(11, [20, 0, 1])], [3], 8, 2, torch.bfloat16, seed=5)
    used = np.zeros((c.n, BS), bool)
    for i in range(c.B):
        for t in range(int(c.lens[i])):
            used[c.tables[i, t // BS], t % BS] = True
    for x in (c.pool.k, c.pool.v):
        x.transpose(1, 2)[torch.from_numpy(~used).cuda()] = float("nan")
    out = c.call()
    ok(pa, c.pool)
    k, v = c.pool.k.nan_to_num(), c.pool.v.nan_to_num()
    c.pool.k.copy_(k); c.pool.v.copy_(v)
    c.check(out)
    c.pool.close()


def test_nan_reaches_the_rows_that_attend_it_and_no_others(pa):
    """As in the plain decode: a NaN query, a NaN key of a sequence's last
    token, a NaN value of the prefix."""
    c = Shared(pa, [(12, [20, 40, 0, 500])], [30], 8, 2, torch.bfloat16, seed=11)
    i, j = int(c.members[0]), int(c.members[1])
    clean = c.call()
    c.q[i, 3] = float("nan")
    out = c.call()
    assert torch.isnan(out[i, 3]).all()
    out[i, 3] = clean[i, 3]
    assert torch.equal(out, clean)
    c.q[i, 3] = 0.5
    clean = c.call()
    t = int(c.lens[j]) - 1
    c.pool.k[int(c.tables[j, t // BS]), 1, t % BS] = float("nan")
    out = c.call()
    # (a sequence whose whole cache is the prefix ends in a token of every member)
    seen = torch.tensor(c.members.tolist() if t < 12 * BS else [j], device="cuda")
    assert torch.isnan(out[seen, 4:]).all()
    out[seen, 4:] = clean[seen, 4:]
    assert torch.equal(out, clean)
    c.pool.k[int(c.tables[j, t // BS]), 1, t % BS] = 0.5
    clean = c.call()
    c.pool.v[int(c.tables[i, 2]), 0, 5, 7] = float("nan")
    out = c.call()
    m = torch.from_numpy(c.members).long().cuda()
    assert torch.isnan(out[m, :4, 7]).all()
    out[m, :4, 7] = clean[m, :4, 7]
    assert torch.equal(out, clean)
    ok(pa, c.pool)
    c.pool.close()


@pytest.mark.parametrize("spare_width", [1, 9000, 9001, 9002])
def test_broken_groups_are_reported_and_ignored(pa, spare_width):
    """(Wide tables are checked by a cluster, four entries at a time when rows allow it.)"""
    c = Shared(pa, [(4, [20, 5, 1]), (6, [30, 2])], [100], 8, 2, torch.bfloat16, seed=6, spare_width=spare_width)
    i32 = lambda x: cuda(np.array(x, np.int32))  # noqa: E731
    m, s = c.members.tolist(), c.start.tolist()
    other = int(np.argmax(c.lens))
    for change in [dict(prefix_blocks=i32([5, 6])),                      # one block too many
                   dict(prefix_blocks=i32([4, -1])), dict(prefix_blocks=i32([4, 1 << 20])),
                   dict(members=i32([m[0], m[1], m[0], m[3], m[4]])),    # twice in one group
                   dict(members=i32([m[0], m[1], m[2], m[3], m[0]])),    # in two groups
                   dict(members=i32([m[0], m[1], m[2], m[3], c.B])), dict(members=i32([-1] + m[1:])),
                   dict(members=i32([m[0], m[1], other] + m[3:])),       # other blocks
                   dict(group_start=i32([0, 3, 4])), dict(group_start=i32([1, 3, 5])), dict(group_start=i32([0, 5, 5])),
                   dict(group_start=i32([0, 7, 5])), dict(group_start=i32([0, -3, 5]))]:
        out = c.call(**change)
        code, _ = pa.pa_check(c.pool)
        assert code == pa.PA_ERR_DEVICE_CHECK, change
        c.check(out)
    assert s == [0, 3, 5]
    out = c.call()
    ok(pa, c.pool)
    c.check(out)
    c.pool.close()


def test_bad_blocks_are_skipped(pa):
    """A block out of range in the shared part is left out for every member, as pa_decode leaves it out."""
    c = Shared(pa, [(20, [20] * 40), (8, [3, 3])], [], 8, 2, torch.bfloat16, seed=7)
    t = c.tables.copy()
    for i in c.members[:40]:
        t[i, 3] = c.n
        t[i, 8:16] = -4         # a whole chunk
    for i in c.members[40:]:
        t[i, :8] = -1           # a whole prefix
    out = c.call(block_tables=cuda(t))
    assert pa.pa_check(c.pool)[0] == pa.PA_ERR_DEVICE_CHECK
    plain = torch.empty_like(out)
    pa.pa_decode_split(c.pool, c.q, cuda(t), cuda(c.lens), D ** -0.5, plain)
    assert pa.pa_check(c.pool)[0] == pa.PA_ERR_DEVICE_CHECK
    assert torch.allclose(out, plain, atol=1e-4, rtol=1e-4)
    c.pool.close()


def test_lengths_out_of_range(pa):
    c = Shared(pa, [(4, [20, 5])], [30], 8, 2, torch.bfloat16, seed=8)
    L = c.lens.copy()
    L[int(c.members[0])] = c.tables.shape[1] * BS + 1
    out = c.call(seq_lens=cuda(L))
    assert pa.pa_check(c.pool)[0] == pa.PA_ERR_DEVICE_CHECK
    c.check(out, rows=[i for i in range(c.B) if i != int(c.members[0])])
    L[int(c.members[0])] = -1
    out = c.call(seq_lens=cuda(L))
    assert pa.pa_check(c.pool)[0] == pa.PA_ERR_DEVICE_CHECK
    assert (out[int(c.members[0])] == 0).all()
    c.pool.close()


def test_same_bits_every_time_graph_and_stream(pa):
    c = Shared(pa, [(60, [40] * 50)], [500, 2], 8, 2, torch.bfloat16, seed=9)
    ref = c.call()
    for _ in range(5):
        assert torch.equal(c.call(), ref)
    dev = dict(block_tables=cuda(c.tables), seq_lens=cuda(c.lens), group_start=cuda(c.start), members=cuda(c.members),
               prefix_blocks=cuda(c.prefix))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(ref)
    pa.pa_decode_shared(c.pool, c.q, scale=D ** -0.5, out=out, stream=s, **dev)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, ref)
    ws = pa.shared_workspace_for(c.pool, c.q, dev["block_tables"], dev["prefix_blocks"])
    ws.fill_(0xff)   # its contents do not matter
    graphs, outs = [], [torch.empty_like(ref), torch.empty_like(ref)]
    for o in outs:   # two graphs that share the workspace, replayed in order
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_decode_shared(c.pool, c.q, scale=D ** -0.5, out=o, workspace=ws, **dev)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
    ok(pa, c.pool)
    c.pool.close()


def test_largest_batch(pa):
    """4,096 sequences behind one block, groups of 2,048."""
    c = Shared(pa, [(9, [1] * 2048), (3, [2] * 2048)], [], 2, 1, torch.float16, seed=10)
    out = c.call()
    ok(pa, c.pool)
    c.check(out, rows=range(0, c.B, 97))
    c.pool.close()


def test_refusals(pa):
    pool = pa.Pool(4, 2, torch.bfloat16)
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    good = dict(q=z(2, 4, D, t=torch.bfloat16), block_tables=z(2, 2), seq_lens=z(2), scale=0.1,
                out=z(2, 4, D, t=torch.float32), group_start=torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
                members=torch.tensor([0, 1], dtype=torch.int32, device="cuda"), prefix_blocks=z(1))
    pa.pa_decode_shared(pool, **good)
    ok(pa, pool)
    for change, error in [(dict(members=z(3)), pa.PagedAttentionError), (dict(members=z(0)), pa.PagedAttentionError),
                          (dict(group_start=z(3)), ValueError), (dict(members=z(2, t=torch.int64)), TypeError),
                          (dict(q=z(2, 18, D, t=torch.bfloat16), out=z(2, 18, D, t=torch.float32)), pa.PagedAttentionError),
                          (dict(out=z(2, 4, D, t=torch.float64)), ValueError),
                          (dict(workspace=z(4096, t=torch.uint8)), pa.PagedAttentionError),
                          (dict(scale=float("nan")), pa.PagedAttentionError), (dict(scale=float("inf")), pa.PagedAttentionError),
                          (dict(members=torch.zeros(2, dtype=torch.int32)), ValueError)]:
        with pytest.raises(error):
            pa.pa_decode_shared(pool, **{**good, **change})
    many = dict(q=z(4097, 2, D, t=torch.bfloat16), block_tables=z(4097, 1), seq_lens=z(4097),
                out=z(4097, 2, D, t=torch.float32))
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_decode_shared(pool, **{**good, **many})
    pool.close()
