"""Waits of the 8-bit decode that run out: some loads are held back, every warp leaves within the limit, the error is
reported, the rows that it concerns are NaN and no others, and the context goes on."""
import numpy as np
import pytest
import torch

from ._ops import D, cuda
from ._ops8 import ok8
from .test_gpu_decode8 import SCALE, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


def held(c, cta, limit=20_000_000, out_dtype=torch.float32, workspace=None):
    out = torch.full((len(c.lens), c.Hq, D), 7.0, dtype=out_dtype, device="cuda")
    status = c.pa.pa_selftest_decode8_timeout(c.pool, c.q, cuda(c.tables), cuda(np.asarray(c.lens, np.int32)), SCALE, out,
                                              limit, cta, workspace)
    return status, out


def segments(out, c):
    """[B][Hkv]: 1 where the rows of a kv head's group are NaN throughout; all or none of them are."""
    nan = torch.isnan(out).view(len(c.lens), c.Hkv, -1)
    assert torch.equal(nan.any(2), nan.all(2))
    return nan.all(2)


PLANS = [  # a CTA a segment; equal ranges: many segments a CTA, several CTAs a segment, both
    ([40, 0, 300, 16, 1], 8, 2, None), ([500] * 40, 16, 2, 40), ([30, 0, 17, 200, 1, 90] * 40, 8, 2, None),
    ([9000], 6, 1, None), ([30000, 0, 5, 17000, 900], 12, 2, None), ([4000, 700, 2000] * 4, 40, 40, None),
]


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("lens,Hq,Hkv,width", PLANS)
def test_all_loads_that_do_not_come(pa, kind, lens, Hq, Hkv, width):
    c = Case(pa, lens, Hq, Hkv, kind, seed=60, width=width)
    want = c.call()
    ok8(pa, c.pool)
    for out_dtype in (torch.float32, torch.bfloat16):
        status, out = held(c, -1, out_dtype=out_dtype)
        assert status == pa.PA_OK
        assert pa.pa_check8(c.pool)[0] == pa.PA_ERR_TIMEOUT
        lens_ = torch.tensor(lens, device="cuda")
        assert segments(out, c)[lens_ > 0].all()
        assert (out[lens_ == 0] == 0).all(), "the rows of empty sequences wait for nothing"
    assert torch.equal(c.call(), want)
    ok8(pa, c.pool)


@pytest.mark.parametrize("cta", [0, 3, 77, 151])
@pytest.mark.parametrize("lens,Hq,Hkv,width", PLANS)
def test_loads_of_one_cta_that_do_not_come(pa, cta, lens, Hq, Hkv, width):
    """Only the rows of segments in that CTA's range are lost, whatever the workspace held."""
    c = Case(pa, lens, Hq, Hkv, "int8", seed=61, width=width)
    want = c.call()
    ws = pa.decode8_workspace_for(c.pool, c.q, cuda(c.tables))
    ws.fill_(0xff if cta % 2 else 0x3f)
    status, out = held(c, cta, workspace=ws)
    assert status == pa.PA_OK
    code = pa.pa_check8(c.pool)[0]
    nan = segments(out, c)
    assert code == (pa.PA_ERR_TIMEOUT if nan.any() else pa.PA_OK)
    rows = nan.repeat_interleave(Hq // Hkv, 1)
    assert torch.equal(out[~rows], want[~rows])
    assert not nan[torch.tensor(lens, device="cuda") == 0].any()
    units = (sum(1 + -(-x // 16) for x in lens if x)) * Hkv  # a start and the tiles of each segment
    if max(lens) > 97 * 16:  # equal ranges: at most what one range holds, with what its ends cut
        per = max(8, -(-units // 152))
        assert int(nan.sum()) <= per // 2 + 2
        if cta * per + 2 < units:
            assert nan.any(), "a range of at least two units has a tile"
    assert torch.equal(c.call(workspace=ws), want)
    ok8(pa, c.pool)


def test_short_limits_and_limits_out_of_range(pa):
    c = Case(pa, [700, 90], 8, 2, "e4m3", seed=62)
    want = c.call()
    for limit in (0, -1, 1_000_000_001):
        assert held(c, -1, limit)[0] == pa.PA_ERR_INVALID
    for cta in (-2, 1 << 16):
        assert held(c, cta)[0] == pa.PA_ERR_INVALID
    ok8(pa, c.pool)
    status, out = held(c, 65535)  # no such CTA: nothing is held
    assert status == pa.PA_OK and torch.equal(out, want)
    ok8(pa, c.pool)
    status, out = held(c, -1, 1)  # every wait that does not end at once
    assert status == pa.PA_OK and pa.pa_check8(c.pool)[0] == pa.PA_ERR_TIMEOUT
    assert segments(out, c).all()
    assert torch.equal(c.call(), want)
    ok8(pa, c.pool)
