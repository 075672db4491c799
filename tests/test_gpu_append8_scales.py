"""Blocks that hold the largest scales: a run that goes on with one keeps it, to the last exponent (2^127)."""
import numpy as np
import pytest
import torch

from ._ops import BS, cuda, to64
from ._ops8 import KINDS, fill8, ok8, raw, type8, write8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


@pytest.mark.parametrize("kind", KINDS)
def test_blocks_with_the_largest_scales(pa, kind):
    rng = np.random.default_rng(1)
    exps = np.array([250, 251, 252, 253, 254, 255], np.uint8)
    nb, hkv = len(exps), 2
    pool = pa.Pool8(nb, hkv, type8(kind))
    zero = np.zeros((nb, hkv, BS, 128), np.uint8)
    e = np.repeat(exps[:, None], hkv, 1)
    fill8(pool, zero, zero, e, e)
    slots = (np.arange(nb) * BS + 3).astype(np.int64)
    kn, vn = ((torch.from_numpy(rng.uniform(-1, 1, (nb, hkv, 128))) * 3.3e38).to(torch.bfloat16).cuda() for _ in "kv")
    pa.pa_cache_append8(pool, kn, vn, cuda(slots))
    k, ek = write8(zero, e, to64(kn), slots, kind)
    v, ev = write8(zero, e, to64(vn), slots, kind)
    got = raw(pool)
    for x in (0, 1):  # (codes under the exponent of NaN do not count)
        got[x][5] = (k, v)[x][5]
    for g, ref in zip(got, (k, v, ek, ev)):
        assert np.array_equal(g, ref)
    assert (np.abs(got[0][4, :, 3].view(np.int8)) > 0).any()
    ok8(pa, pool)
