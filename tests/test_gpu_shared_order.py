"""Shared-prefix decode where the hand-overs inside the prefix product matter:
maxima that move in every chunk, calls on two streams at once, a workspace of
exactly the size asked for."""
import numpy as np
import pytest
import torch

from ._ops import D, cuda, ok
from .test_gpu_shared import Shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("members", [4, 20, 34, 64])
def test_maxima_that_move_in_every_chunk(pa, members, out_dtype, dtype):
    """Keys grow by 0.35 a block along the prefix: the maximum of about 100
    scores a chunk grows by 0.35 * 8 * 2.5 of their spread, 10 log2 units, so
    the output so far is rescaled before every value product (members: rows
    of one tile, and of two), and every dim of it has to be rescaled before the
    product adds to it."""
    c = Shared(pa, [(120, [3] * members)], [], 8, 2, dtype, seed=40)
    first = c.tables[c.members[0]]
    at = torch.from_numpy(first[:120].astype(np.int64)).cuda()
    c.pool.k[at] *= (0.35 * torch.arange(120, device="cuda", dtype=torch.float32)).view(-1, 1, 1, 1).to(dtype)
    ref = c.call(out_dtype)
    ok(pa, c.pool)
    c.check(ref, rows=range(0, c.B, 5))
    for _ in range(20):
        assert torch.equal(c.call(out_dtype), ref)
    ok(pa, c.pool)
    c.pool.close()


def test_two_streams_at_once(pa):
    """Two calls in flight together, a workspace each: the bits of a call alone."""
    c = Shared(pa, [(90, [40] * 40), (16, [7, 300])], [500, 2], 8, 2, torch.bfloat16, seed=41)
    ref = c.call()
    dev = dict(block_tables=cuda(c.tables), seq_lens=cuda(c.lens), group_start=cuda(c.start), members=cuda(c.members),
               prefix_blocks=cuda(c.prefix))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [pa.shared_workspace_for(c.pool, c.q, dev["block_tables"], dev["prefix_blocks"]) for _ in streams]
    outs = [[torch.full_like(ref, float("nan")) for _ in range(12)] for _ in streams]
    torch.cuda.synchronize()
    for n in range(12):
        for s, w, o in zip(streams, ws, outs):
            pa.pa_decode_shared(c.pool, c.q, scale=D ** -0.5, out=o[n], workspace=w, stream=s, **dev)
    torch.cuda.synchronize()
    for o in outs:
        for x in o:
            assert torch.equal(x, ref)
    ok(pa, c.pool)
    c.pool.close()


@pytest.mark.parametrize("groups,alone,hq,hkv", [([(5, [3] * 64)], [], 4, 1), ([(5, [3] * 65), (9, [1, 2])], [70], 32, 8),
                                                 ([(2, [1, 2])] * 45, [], 5, 1), ([], [10, 700], 8, 2)])
def test_nothing_is_written_past_the_workspace(pa, groups, alone, hq, hkv):
    c = Shared(pa, groups, alone, hq, hkv, torch.bfloat16, seed=42)
    n = pa.lib.pa_decode_shared_workspace_bytes(c.pool.handle, c.B, hq, c.tables.shape[1], len(c.prefix))
    room = torch.full((n + 2 * 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    at = 4096 + -(room.data_ptr() + 4096) % 256
    out = c.call(workspace=room[at:at + n])
    ok(pa, c.pool)
    c.check(out, rows=range(0, c.B, 7))
    assert (room[:at] == 0x5a).all() and (room[at + n:] == 0x5a).all()
    c.pool.close()
