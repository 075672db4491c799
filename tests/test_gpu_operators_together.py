"""The cache operators in one run, as a serving loop uses them: prompts behind a
shared prefix are written with rotary positions of three axes, decode steps
attend the prefix once for the batch, the attention weights are summed, the
cache is cut back by them, and decoding goes on in the closed-up cache.  A
64-bit model of the cache follows along; the allocator's tables drive both."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, attend64, cuda, evict64, half_step, ok, rand16, rope64, to64

pytestmark = pytest.mark.gpu

HQ, HKV, DTYPE = 8, 2, torch.bfloat16
AXES = [f % 3 for f in range(64)]
INV = (10000.0 ** (-np.arange(0, 128, 2) / 128)).astype(np.float32)


class Model:
    """Each sequence's cache as rows: what the pool should hold, bit for bit
    (read back from the pool when written, since the rounding is the kernel's)."""

    def __init__(self):
        self.k, self.v, self.w = {}, {}, {}


def pool_rows(x, table, L):
    blocks = x[torch.tensor(table[:-(-L // BS)], device="cuda")]
    return to64(blocks.transpose(1, 2).reshape(-1, HKV, D)[:L]).transpose(1, 0, 2)


def device_tables(alloc, seqs, width):
    t = np.full((len(seqs), width), -1, np.int32)
    for i, s in enumerate(seqs):
        row = alloc.table(s)
        t[i, :len(row)] = row
    return t


def test_prompts_steps_eviction_and_on():
    import paged_kv_cache_227_gb300 as pa
    torch.cuda.set_device(0)
    rng = np.random.default_rng(17)
    n_blocks, width, prefix, own = 400, 24, 160, [37, 5, 64, 1, 90]
    pool = pa.Pool(n_blocks, HKV, DTYPE)
    alloc = pa.BlockAllocator(n_blocks, free_order=rng.permutation(n_blocks))
    seqs = list(range(5))
    pos_of = {}

    def write(seq_slots, positions):
        """Turns and writes new tokens; returns their turned queries."""
        n = len(seq_slots)
        qkv = rand16(rng, DTYPE, n, HQ + 2 * HKV, D).cuda()
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        qo = torch.empty(n, HQ, D, dtype=DTYPE, device="cuda")
        pos = np.array(positions, np.int32).T.copy()
        pa.pa_rope_append(pool, q, k, v, cuda(pos), cuda(INV), AXES, cuda(np.array(seq_slots, np.int64)), qo)
        want = rope64(to64(k), pos, INV, AXES, False)
        slots = torch.tensor(seq_slots, device="cuda")
        got = to64(pool.k.transpose(1, 2).reshape(-1, HKV, D)[slots])
        mag = np.abs(to64(k))
        mag = mag[..., :64] + mag[..., 64:]
        mag = np.concatenate([mag, mag], -1)
        assert (np.abs(got - want) <= half_step(DTYPE) * (np.abs(want) + 2e-6 * mag) + 2e-6 * mag).all()
        return qo

    # the shared prompt, then each sequence's own
    alloc.seq_add(99)
    slots, _ = alloc.extend(99, prefix)
    write(slots.tolist(), [(t // 8, t % 8, t % 5) for t in range(prefix)])
    for s, n in zip(seqs, own):
        alloc.fork(99, s)
        slots, _ = alloc.extend(s, n)
        write(slots.tolist(), [(20 + t, t, 0) for t in range(n)])
        pos_of[s] = 20 + n
    weights = torch.zeros(5, HKV, width * BS, device="cuda")
    sums = np.zeros((5, HKV, width * BS))
    scale = D ** -0.5

    def step(shared):
        slots, pos = [], []
        for s in seqs:
            slot, src, dst = alloc.append_slot(s)
            if src >= 0:
                pa.pa_copy_blocks(pool, torch.tensor([src], dtype=torch.int32, device="cuda"),
                                  torch.tensor([dst], dtype=torch.int32, device="cuda"))
            slots.append(slot)
            pos.append((pos_of[s], 0, 0))
            pos_of[s] += 1
        q = write(slots, pos)
        tables = device_tables(alloc, seqs, width)
        lens = np.array([alloc.seq_len(s) for s in seqs], np.int32)
        bt, sl = cuda(tables), cuda(lens)
        out = torch.empty(5, HQ, D, device="cuda")
        pa.pa_decode_weights(pool, q, bt, sl, scale, out, weights)
        for i, s in enumerate(seqs):
            L = int(lens[i])
            ref, p = attend64(to64(q[i]), pool_rows(pool.k, tables[i].tolist(), L), pool_rows(pool.v, tables[i].tolist(), L),
                              scale)
            assert np.abs(to64(out[i]) - ref).max() < 1e-4
            sums[i, :, :L] += p.reshape(HKV, HQ // HKV, L).sum(1)
        assert np.abs(to64(weights) - sums).max() < 1e-3
        if shared:
            gs, mem, pre = pa.cascade_groups(tables, lens, HQ, HKV, max_members=5)
            assert len(pre) == 1 and pre[0] == prefix // BS and len(mem) == 5
            again = torch.empty_like(out)
            pa.pa_decode_shared(pool, q, bt, sl, scale, again, cuda(gs), cuda(mem), cuda(pre))
            assert (again - out).abs().max() < 1e-4
        ok(pa, pool)

    for _ in range(3):
        step(shared=True)

    # cut back to at most 100 tokens each: the shared blocks are replaced, the others stay
    old = device_tables(alloc, seqs, width)
    lens = np.array([alloc.seq_len(s) for s in seqs], np.int32)
    keep = np.array([100, 100, 120, 30, 10 ** 6], np.int32)
    keys = [pool_rows(pool.k, old[i].tolist(), int(lens[i])) for i in range(5)]
    vals = [pool_rows(pool.v, old[i].tolist(), int(lens[i])) for i in range(5)]
    parent = pool_rows(pool.k, alloc.table(99), prefix)
    alloc.evict(seqs, keep.tolist())
    new = device_tables(alloc, seqs, width)
    before = weights.cpu().numpy().copy()
    n_out = torch.zeros(5, dtype=torch.int32, device="cuda")
    kept = torch.zeros(5, HKV, width * BS, dtype=torch.int32, device="cuda")
    pa.pa_evict(pool, weights, cuda(old), cuda(lens), cuda(keep), n_out, kept, n_sink=4, n_recent=16, dst_tables=cuda(new))
    ok(pa, pool)
    for i, s in enumerate(seqs):
        n = int(n_out[i])
        assert n == min(int(keep[i]), int(lens[i])) == alloc.seq_len(s)
        k1, v1 = pool_rows(pool.k, new[i].tolist(), n), pool_rows(pool.v, new[i].tolist(), n)
        for h in range(HKV):
            at = evict64(before[i, h], int(lens[i]), int(keep[i]), 4, 16)
            assert kept[i, h, :n].cpu().numpy().tolist() == at.tolist()
            assert np.array_equal(k1[h], keys[i][h][at]) and np.array_equal(v1[h], vals[i][h][at])
            sums[i, h, :n] = sums[i, h, at]
            sums[i, h, n:] = 0
    assert np.array_equal(parent, pool_rows(pool.k, alloc.table(99), prefix)), "the parent's blocks are untouched"
    for _ in range(2):
        step(shared=False)
    pool.close()


def test_top_blocks_of_a_large_pool():
    """Offsets past 2^32 bytes (4.6 GB an array): each operator gives the bits
    that it gives at the bottom of the pool."""
    import paged_kv_cache_227_gb300 as pa
    torch.cuda.set_device(0)
    N, hkv, hq, L = 140000, 8, 16, 150
    pool = pa.Pool(N, hkv, DTYPE)
    n = -(-L // BS)
    results = []
    for base in (0, N - 64):
        rng = np.random.default_rng(23)
        perm = base + rng.permutation(64).astype(np.int32)
        shared, rest = perm[:4], perm[4:]
        tables = np.stack([np.concatenate([shared, rest[i * (n - 4):(i + 1) * (n - 4)]]) for i in range(3)]).astype(np.int32)
        fresh = rest[3 * (n - 4):3 * (n - 4) + 9].reshape(3, 3)
        slots = np.concatenate([t.astype(np.int64)[:, None] * BS + np.arange(BS) for t in tables]).reshape(3, -1)[:, :L]
        qkv = rand16(rng, DTYPE, 3 * L, hq + 2 * hkv, D).cuda()
        # the shared blocks hold one prompt: every sequence writes the same rows there
        qkv.view(3, L, -1)[:, :64] = qkv.view(3, L, -1)[0, :64].clone()
        pos = np.tile(np.arange(L), 3).astype(np.int32)[None]
        qo = torch.empty(3 * L, hq, D, dtype=DTYPE, device="cuda")
        pa.pa_rope_append(pool, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], cuda(pos), cuda(INV), [0] * 64,
                          cuda(slots.reshape(-1)), qo)
        q = qo.view(3, L, hq, D)[:, -1].contiguous()
        bt, sl = cuda(tables), cuda(np.full(3, L, np.int32))
        out, again = torch.empty(3, hq, D, device="cuda"), torch.empty(3, hq, D, device="cuda")
        w = torch.zeros(3, hkv, n * BS, device="cuda")
        pa.pa_decode_weights(pool, q, bt, sl, D ** -0.5, out, w)
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        pa.pa_decode_shared(pool, q, bt, sl, D ** -0.5, again, i32(0, 3), i32(0, 1, 2), i32(4))
        kept = torch.zeros(3, hkv, n * BS, dtype=torch.int32, device="cuda")
        n_out = i32(0, 0, 0)
        summed = w.clone()
        pa.pa_evict(pool, w, bt, sl, i32(40, 41, 48), n_out, kept, n_sink=2, n_recent=8, dst_tables=cuda(fresh))
        ok(pa, pool)
        at = torch.from_numpy(fresh.astype(np.int64)).cuda()
        results.append([x.clone() for x in (qo, out, again, summed, w, kept, n_out, pool.k[at][:, :2], pool.v[at][:, :2])])
        assert (out - again).abs().max() < 1e-4
    for a, b in zip(*results):
        assert torch.equal(a, b)
    pool.close()
