"""Waits of the prefix product that run out: its loads are held back, every warp
of it leaves within the limit, the error is reported and the context goes on."""
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


def arguments(c):
    return dict(block_tables=cuda(c.tables), seq_lens=cuda(c.lens), group_start=cuda(c.start), members=cuda(c.members),
                prefix_blocks=cuda(c.prefix), scale=D ** -0.5)


@pytest.mark.parametrize("groups", [[(1, [3, 4])], [(20, [5] * 3), (9, [1, 2])], [(40, [9] * 70)]])
def test_waits_that_run_out_are_reported(pa, groups):
    """One chunk for one team, chunks in turn, two tiles and several pieces a CTA."""
    c = Shared(pa, groups, [30], 8, 2, torch.bfloat16, seed=50)
    ref = c.call()
    ok(pa, c.pool)
    out = torch.empty_like(ref)
    assert pa.pa_selftest_shared_timeout(c.pool, c.q, out=out, limit_ns=20_000_000, **arguments(c)) == pa.PA_OK
    assert pa.pa_check(c.pool)[0] == pa.PA_ERR_TIMEOUT
    alone = int(np.setdiff1d(np.arange(c.B), c.members)[0])
    assert torch.equal(out[alone], ref[alone]), "a sequence in no group does not wait for the product"
    assert torch.equal(c.call(), ref)
    ok(pa, c.pool)
    c.pool.close()


def test_limits_out_of_range_are_refused(pa):
    c = Shared(pa, [(1, [3, 4])], [], 4, 1, torch.float16, seed=51)
    out = torch.empty(c.B, 4, D, device="cuda")
    for limit in (0, -1, 1_000_000_001):
        assert pa.pa_selftest_shared_timeout(c.pool, c.q, out=out, limit_ns=limit, **arguments(c)) == pa.PA_ERR_INVALID
    ok(pa, c.pool)
    c.pool.close()
