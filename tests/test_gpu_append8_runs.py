"""Two runs of one call in one block.  A block's rows have to be one run; where they are not, one run at most is
written into each of the block's tiles, whole, the others are skipped, and that is reported.  So a tile holds what it
held, or what the definition gives for one of its runs alone, byte for byte: no row of an earlier call is lost."""
import numpy as np
import pytest
import torch

from ._ops import BS, cuda, to64
from ._ops8 import KINDS, fill8, filled_pool8, ok8, rand_rows, raw, runs_of, write8
from .test_gpu_append8 import same, slots_for
from .test_gpu_norm_rope import Tokens, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


def by_token(held, new):
    """Rows in the order of the tokens: the first new one of each sequence, then the second; block i is sequence i's."""
    return np.concatenate([np.arange(len(held)) * BS + np.asarray(held) + j for j in range(new)]).astype(np.int64)


CALLS = {
    "two sequences by token": by_token([5, 3], 2),
    "the first tokens of blocks, by token": by_token([0, 0, 0], 3),
    "more sequences than a window, by token": by_token([(5 * i) % 13 for i in range(40)], 3),
    "four hundred sequences by token": by_token([(7 * i) % 15 for i in range(400)], 2),
    "a slot twice": np.array([37, 90, 37], np.int64),
    "a slot twice on end": np.array([37, 37], np.int64),
    "backwards": np.array([9, 8, 7, 6], np.int64),
    "padding inside a block": np.array([4, 5, -1, 7, 8, 33], np.int64),
    "afresh, then behind it": np.array([0, 1, 20, 5, 6], np.int64),
    "behind it, then afresh": np.array([5, 6, 20, 0, 1], np.int64),
    "a window's last row and the next one's": np.concatenate([np.arange(100, 116) * BS, [99 * BS, 115 * BS + 4]]).astype(np.int64),
    "a thousand rows apart": np.concatenate([[3], np.arange(BS, 1000 + BS), [9, 10]]).astype(np.int64),
}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", CALLS)
def test_a_block_of_two_runs(pa, name, kind):
    rng = np.random.default_rng(len(name))
    slots, hkv = CALLS[name], 3
    nb = int(slots.max()) // BS + 2
    pool, start = filled_pool8(pa, rng, kind, nb, hkv, spread=6)
    n = len(slots)
    # rows of all sizes, so that scales grow, by different powers
    kn, vn = ((rand_rows(rng, torch.float32, n, hkv) * torch.from_numpy(
        2.0 ** rng.integers(-3, 9, (n, 1, 1))).cuda()).to(torch.bfloat16) for _ in "kv")
    pa.pa_cache_append8(pool, kn, vn, cuda(slots))
    code, slot = pa.pa_check8(pool)
    assert code == pa.PA_ERR_DEVICE_CHECK
    runs = runs_of(slots, nb * BS)
    of = {}
    for r in runs:
        of.setdefault(int(slots[r[0]]) // BS, []).append(r)
    twice = {b for b, rs in of.items() if len(rs) > 1}
    assert slot in {int(slots[r[0]]) for b in twice for r in of[b]}, "the detail is the first slot of such a run"
    got = raw(pool)
    for x, rows in ((0, to64(kn)), (1, to64(vn))):
        codes, exps = start[x], start[2 + x]
        alone = [r for r in runs if int(slots[r[0]]) // BS not in twice]
        at = np.concatenate(alone + [[]]).astype(int)
        want, we = write8(codes, exps, rows[at], slots[at], kind) if len(at) else (codes, exps)
        rest = np.setdiff1d(np.arange(nb), list(twice))
        assert np.array_equal(got[x][rest], want[rest]) and np.array_equal(got[2 + x][rest], we[rest])
        for b in twice:
            can = [(codes[b], exps[b])]
            for r in of[b]:
                c, e = write8(codes[b:b + 1], exps[b:b + 1], rows[r], slots[r] - b * BS, kind)
                can.append((c[0], e[0]))
            for h in range(hkv):
                assert any(np.array_equal(got[x][b, h], c[h]) and got[2 + x][b, h] == e[h] for c, e in can), (b, h)
    # the next call on the same blocks is an ordinary one
    fill8(pool, *start)
    first = slots[[r[0] for r in runs if r is of[int(slots[r[0]]) // BS][0]]]
    kn, vn = kn[:len(first)].contiguous(), vn[:len(first)].contiguous()
    pa.pa_cache_append8(pool, kn, vn, cuda(first))
    k, ek = write8(start[0], start[2], to64(kn), first, kind)
    v, ev = write8(start[1], start[3], to64(vn), first, kind)
    same(pool, (k, v, ek, ev))
    ok8(pa, pool)


@pytest.mark.parametrize("kind", KINDS)
def test_batches_in_any_order_step_after_step(pa, kind):
    """Sequences that change their rows of the call from step to step, some with several tokens: never reported."""
    rng = np.random.default_rng(20)
    B, hkv = 45, 2
    pool, (k, v, ek, ev) = filled_pool8(pa, rng, kind, 4 * B, hkv)
    held, tables = rng.integers(0, 20, B), rng.permutation(4 * B).reshape(B, 4)
    for step in range(6):
        slots = []
        for i in rng.permutation(B)[:int(rng.integers(5, B + 1))]:
            p = held[i] + np.arange(int(rng.integers(1, 6)))
            held[i] += len(p)
            slots.append(tables[i, p // BS] * BS + p % BS)
        slots = np.concatenate(slots).astype(np.int64)
        kn, vn = rand_rows(rng, torch.float16, len(slots), hkv), rand_rows(rng, torch.float16, len(slots), hkv)
        pa.pa_cache_append8(pool, kn, vn, cuda(slots))
        k, ek = write8(k, ek, to64(kn), slots, kind)
        v, ev = write8(v, ev, to64(vn), slots, kind)
        same(pool, (k, v, ek, ev))
    ok8(pa, pool)


def test_two_runs_on_the_way_through_norms(pa):
    """The query rows of tokens that keep out of the cache are written all the same."""
    rng = np.random.default_rng(21)
    slots = by_token([2, 9, 4], 2)
    t = Tokens(rng, len(slots), 8, 2, torch.bfloat16, 128, 1, False)
    w = weight(rng, torch.bfloat16)
    pool, start = filled_pool8(pa, rng, "e4m3", 4, 2)
    pa.pa_norm_rope_append8(pool, *t.args(w, w, np.concatenate(slots_for(rng, 4, [(3, 6)]))))
    ok8(pa, pool)
    want = t.q_out.clone()
    t.q_out.fill_(float("nan"))
    fill8(pool, *start)
    pa.pa_norm_rope_append8(pool, *t.args(w, w, slots))
    assert pa.pa_check8(pool)[0] == pa.PA_ERR_DEVICE_CHECK
    assert torch.equal(t.q_out, want)
    got = raw(pool)
    assert np.array_equal(got[0][3], start[0][3]) and np.array_equal(got[1][3], start[1][3])
    for b, off in enumerate((2, 9, 4)):
        held = np.setdiff1d(np.arange(BS), [off, off + 1])
        for h in range(2):
            if got[3][b, h] == start[3][b, h]:
                assert np.array_equal(got[1][b, h, held], start[1][b, h, held])
