"""Host side of the cache operators: refusals that need no GPU, and the block
tables that an eviction gets."""
import ctypes
import types

import numpy as np
import pytest
import torch

import paged_kv_cache_227_gb300 as pa

from ._ops import evict64


def fake_pool(dtype=torch.bfloat16, n_kv_heads=2):
    return types.SimpleNamespace(handle=None, dtype=dtype, n_kv_heads=n_kv_heads, device=torch.device("cuda", 0))


def test_host_tensors_are_refused():
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    q, kv = torch.zeros(3, 4, 128, dtype=bf), torch.zeros(3, 2, 128, dtype=bf)
    with pytest.raises(ValueError, match="must be on the GPU"):
        pa.pa_rope_append(fake_pool(), q, kv, kv, torch.zeros(1, 3, dtype=i32), torch.zeros(64, dtype=f32), [0] * 64,
                          torch.zeros(3, dtype=torch.int64), q)
    w = torch.zeros(3, 2, 32, dtype=f32)
    with pytest.raises(ValueError, match="must be on the GPU"):
        pa.pa_decode_weights(fake_pool(), q, torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32), 0.1, q.float(), w)
    with pytest.raises(ValueError, match="must be on the GPU"):
        pa.pa_evict(fake_pool(), w, torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(3, dtype=i32),
                    torch.zeros(3, dtype=i32), torch.zeros(3, 2, 32, dtype=i32))


def test_null_pools_are_refused():
    assert pa.lib.pa_rope_append(None, None, 0, 1, None, 0, None, 0, None, 1, None, None, 128, 0, None, 1, None, 0,
                                 None) == pa.PA_ERR_INVALID
    assert pa.lib.pa_decode_weights_workspace_bytes(None, 1, 1, 1) == 0
    assert pa.lib.pa_decode_weights(None, None, None, 1, None, 1, 8, 1.0, None, 2, None, 1.0, None, 0,
                                    None) == pa.PA_ERR_INVALID
    assert pa.lib.pa_evict(None, None, None, None, 1, None, 0, None, None, 1, 0, 0, None, None, None) == pa.PA_ERR_INVALID
    assert pa.lib.pa_alloc_evict(None, None, None, 0) == pa.PA_ERR_INVALID


def held(a):
    return sum(a.refcount(b) > 0 for b in range(a.num_blocks))


def test_eviction_tables_of_one_sequence():
    a = pa.BlockAllocator(8, free_order=range(8))
    a.seq_add(0)
    for _ in range(70):
        a.append_slot(0)
    assert a.table(0) == [0, 1, 2, 3, 4]
    a.evict([0], [33])
    assert a.table(0) == [0, 1, 2] and a.seq_len(0) == 33 and a.num_free() == 5
    assert a.append_slot(0)[0] == 2 * 16 + 1, "the next token goes behind the kept ones"
    a.evict([0], [100])
    assert a.table(0) == [0, 1, 2] and a.seq_len(0) == 34, "nothing to evict"
    a.evict([0], [0])
    assert a.table(0) == [] and a.num_free() == 8
    a.evict([], [])


def test_shared_blocks_are_replaced_and_the_sharer_keeps_its_own():
    a = pa.BlockAllocator(10, free_order=range(10))
    a.seq_add(0)
    for _ in range(40):
        a.append_slot(0)      # blocks 0, 1, 2
    a.fork(0, 1)
    a.append_slot(1)          # copy on write: block 3 instead of 2
    a.evict([1], [20])
    assert a.table(1) == [4, 5] and a.table(0) == [0, 1, 2]
    assert [a.refcount(b) for b in range(6)] == [1, 1, 1, 0, 1, 1]


def test_sharers_evicted_in_one_call_both_leave_the_shared_blocks():
    """Neither may write in place what the other still reads, and a block that
    the call releases is not handed to the other."""
    a = pa.BlockAllocator(7, free_order=range(7))
    a.seq_add(0)
    for _ in range(48):
        a.append_slot(0)
    a.fork(0, 1)
    old = set(a.table(0))
    a.evict([0, 1], [32, 17])
    t0, t1 = a.table(0), a.table(1)
    assert len(t0) == 2 and len(t1) == 2 and not (set(t0) | set(t1)) & old and not set(t0) & set(t1)
    assert held(a) == 4 and a.num_free() == 3


def test_errors_change_nothing():
    a = pa.BlockAllocator(4, free_order=range(4))
    a.seq_add(0)
    for _ in range(40):
        a.append_slot(0)
    a.fork(0, 1)
    before = (a.table(0), a.table(1), a.num_free(), a.seq_len(0), a.seq_len(1))
    with pytest.raises(MemoryError):
        a.evict([0, 1], [32, 32])       # 4 new blocks, 1 free
    for seqs, keep in (([0, 9], [1, 1]), ([0, 0], [1, 1]), ([0], [-1])):
        with pytest.raises(pa.PagedAttentionError):
            a.evict(seqs, keep)
    assert before == (a.table(0), a.table(1), a.num_free(), a.seq_len(0), a.seq_len(1))
    with pytest.raises(ValueError):
        a.evict([0], [])
    assert pa.lib.pa_alloc_evict(a._h, None, None, 1) == pa.PA_ERR_INVALID
    assert pa.lib.pa_alloc_evict(a._h, (ctypes.c_int * 1)(0), None, -1) == pa.PA_ERR_INVALID


def test_rewritten_blocks_leave_the_prefix_cache():
    """A block that an eviction rewrites is no longer the prompt it was hashed
    for; released blocks keep their contents and stay findable."""
    a = pa.BlockAllocator(8, free_order=range(8))
    ids = list(range(48))
    a.seq_add(0)
    for x in ids:
        a.append_token(0, x)
    assert a.prefix_stats()[2] == 3
    a.evict([0], [20])
    assert [a.block_hash(b) is not None for b in (0, 1, 2)] == [False, False, True]
    assert a.seq_add_cached(1, ids) == 0, "the chain starts with a rewritten block"
    for x in range(12):
        a.append_token(0, x)
    assert a.block_hash(a.table(0)[1]) is None, "later tokens of an evicted sequence are not hashed"


def test_random_histories_keep_the_counts():
    rng = np.random.default_rng(3)
    a = pa.BlockAllocator(60)
    live = []
    for step in range(600):
        op = rng.integers(0, 4)
        try:
            if op == 0 or not live:
                a.seq_add(step); live.append(step)
            elif op == 1:
                for _ in range(int(rng.integers(1, 30))):
                    a.append_slot(int(rng.choice(live)))
            elif op == 2:
                a.fork(int(rng.choice(live)), step); live.append(step)
            else:
                some = rng.choice(live, size=min(len(live), 3), replace=False)
                a.evict([int(s) for s in some], [int(rng.integers(0, 60)) for _ in some])
        except MemoryError:
            s = live.pop(0)
            a.seq_free(s)
        count = np.zeros(60, int)
        for s in live:
            t = a.table(s)
            assert len(t) == -(-a.seq_len(s) // 16)
            for b in t:
                count[b] += 1
        assert [a.refcount(b) for b in range(60)] == count.tolist()
        assert a.num_free() == int((count == 0).sum())


def test_the_selection_reference_on_small_cases():
    w = np.array([1, 5, 5, 0, 7, 2], np.float32)
    assert evict64(w, 6, 3, 0, 0).tolist() == [1, 2, 4]
    assert evict64(w, 6, 2, 0, 0).tolist() == [1, 4]
    assert evict64(w, 6, 3, 1, 1).tolist() == [0, 4, 5]
    assert evict64(np.array([np.nan, -np.inf, 0], np.float32), 3, 2, 0, 0).tolist() == [1, 2]
