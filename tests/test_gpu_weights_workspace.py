"""Decode with weight sums: its workspace is as large as it says, and two calls
on two streams, a workspace each, do not touch one another."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, cuda, filled_pool, ok, rand16, tables_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


def batch(pa, lens, Hq, Hkv, dtype, seed):
    rng = np.random.default_rng(seed)
    tables, _, nb = tables_for(lens, rng)
    pool = filled_pool(pa, rng, nb, Hkv, dtype)
    q = rand16(rng, dtype, len(lens), Hq, D).cuda()
    return pool, q, cuda(tables), cuda(np.array(lens, np.int32)), tables.shape[1] * BS


@pytest.mark.parametrize("lens,Hq,Hkv", [([700, 90, 1, 0], 8, 2), ([33], 7, 1), ([5000, 20], 40, 40), ([16] * 70, 15, 3)])
def test_nothing_is_written_past_the_workspace_or_the_sums(pa, lens, Hq, Hkv):
    pool, q, bt, sl, span = batch(pa, lens, Hq, Hkv, torch.bfloat16, 3)
    n = pa.lib.pa_decode_weights_workspace_bytes(pool.handle, len(lens), Hq, bt.shape[1])
    room = torch.full((n + 2 * 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    at = 4096 + -(room.data_ptr() + 4096) % 256
    sums = torch.full((len(lens) * Hkv * span + 128,), 7.0, device="cuda")
    w = sums[64:-64].view(len(lens), Hkv, span)
    out = torch.empty(len(lens), Hq, D, device="cuda")
    pa.pa_decode_weights(pool, q, bt, sl, D ** -0.5, out, w, decay=0.0, workspace=room[at:at + n])
    ok(pa, pool)
    assert (room[:at] == 0x5a).all() and (room[at + n:] == 0x5a).all()
    assert (sums[:64] == 7).all() and (sums[-64:] == 7).all()
    for i, L in enumerate(lens):
        assert (w[i, :, L:] == 7).all()
        assert L == 0 or torch.allclose(w[i, :, :L].sum(1), torch.full((Hkv,), Hq / Hkv, device="cuda"), rtol=1e-4)
    pool.close()


def test_two_streams_at_once(pa):
    pool, q, bt, sl, span = batch(pa, [3000, 700, 90, 1] * 8, 8, 2, torch.float16, 4)
    B = 32
    ref, one = torch.empty(B, 8, D, device="cuda"), torch.zeros(B, 2, span, device="cuda")
    pa.pa_decode_weights(pool, q, bt, sl, D ** -0.5, ref, one)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    state = [(pa.weights_workspace_for(pool, q, bt), [torch.zeros_like(one) for _ in range(12)],
              [torch.empty_like(ref) for _ in range(12)]) for _ in streams]
    torch.cuda.synchronize()
    for n in range(12):
        for s, (ws, w, o) in zip(streams, state):
            pa.pa_decode_weights(pool, q, bt, sl, D ** -0.5, o[n], w[n], workspace=ws, stream=s)
    torch.cuda.synchronize()
    for _, w, o in state:
        assert all(torch.equal(x, one) for x in w) and all(torch.equal(x, ref) for x in o)
    ok(pa, pool)
    pool.close()
