"""Both sides of the launch rules of the 8-bit decode, the 8-bit write and the norms: a rule chooses the kernel, not the result."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, ok, to64
from ._ops8 import KINDS, ok8, raw, write8
from .test_gpu_append8 import write_and_compare
from .test_gpu_decode8 import Case
from .test_gpu_norm_rope import EPS, Tokens, check, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


@pytest.mark.parametrize("Hq,Hkv,B", [(24, 3, 21), (16, 4, 16), (8, 8, 9), (38, 38, 4), (24, 3, 51)])
@pytest.mark.parametrize("width", [47, 48, 49])
def test_tables_at_the_limit_of_many_segments(pa, Hq, Hkv, B, width):
    """63, 64, 72, 152 and 153 segments, tables of 48 blocks and one less and more, ragged and alike."""
    rng = np.random.default_rng(width + B)
    for alike in (True, False):
        lens = np.full(B, width * BS) if alike else rng.integers(0, width * BS + 1, B)
        c = Case(pa, lens.tolist(), Hq, Hkv, "int8" if alike else "e4m3", seed=B, width=width)
        c.check(c.call())
        ok8(pa, c.pool)


@pytest.mark.parametrize("Hq,Hkv,dtype,rot,interleaved,n", [
    (12, 2, torch.float16, 64, True, 2432), (12, 2, torch.float16, 64, True, 2433), (5, 1, torch.bfloat16, 96, False, 4864),
    (5, 1, torch.bfloat16, 96, False, 4865), (20, 4, torch.bfloat16, 128, False, 1389), (20, 4, torch.bfloat16, 128, False, 1390),
    (32, 4, torch.float16, 128, True, 486), (32, 4, torch.float16, 128, True, 487)])
def test_norms_at_the_switch_to_rows_that_wait(pa, Hq, Hkv, dtype, rot, interleaved, n):
    rng = np.random.default_rng(n)
    nb = -(-n // BS)
    pool = pa.Pool(nb, Hkv, dtype)
    t = Tokens(rng, n, Hq, Hkv, dtype, rot, 2, interleaved, fused=True)
    wq, wk = weight(rng, dtype), weight(rng, dtype)
    slots = rng.permutation(nb * BS)[:n].astype(np.int64)
    pa.pa_norm_rope_append(pool, *t.args(wq, wk, slots), eps=EPS, interleaved=interleaved)
    ok(pa, pool)
    ref, normed = t.want(t.q, wq)
    check(to64(t.q_out), ref, normed, dtype, rot, interleaved)
    rows = to64(pool.k).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)
    ref, normed = t.want(t.k, wk)
    check(rows[slots], ref, normed, dtype, rot, interleaved)
    pool.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hkv,n", [(8, 3040), (8, 3041), (5, 4048), (5, 4065)])
def test_prompts_into_8_bits_at_the_switch_by_k_and_v_rows(pa, kind, hkv, n):
    """760 CTAs and 764, 759 and 765: one prompt that starts inside a block."""
    rng = np.random.default_rng(n)
    nb = n // BS + 2
    table = rng.permutation(nb)
    p = 5 + np.arange(n)
    ok8(pa, write_and_compare(pa, kind, torch.bfloat16, hkv, table[p // BS] * BS + p % BS, nb, n))


@pytest.mark.parametrize("Hq,Hkv,n,norms", [(32, 8, 304, True), (32, 8, 305, True), (12, 2, 810, False), (12, 2, 811, False),
                                            (7, 7, 1216, True), (7, 7, 1217, False)])
def test_prompts_into_8_bits_at_the_switch_by_query_rows(pa, Hq, Hkv, n, norms):
    """Query rows are the 16-bit append's, bit for bit, on both sides; V codes the definition's."""
    rng = np.random.default_rng(n)
    nb = n // BS + 2
    t = Tokens(rng, n, Hq, Hkv, torch.bfloat16, 128, 1, False, fused=True)
    w = weight(rng, torch.bfloat16) if norms else None
    slots = 3 + np.arange(n)
    p8, p16 = pa.Pool8(nb, Hkv, torch.int8), pa.Pool(nb, Hkv, torch.bfloat16)
    _, v, _, ev = raw(p8)
    pa.pa_norm_rope_append8(p8, *t.args(w, w, slots))
    ok8(pa, p8)
    first = t.q_out.clone()
    pa.pa_norm_rope_append(p16, *t.args(w, w, slots))
    assert torch.equal(first, t.q_out)
    v, ev = write8(v, ev, to64(t.v), slots, "int8")
    got = raw(p8)
    assert np.array_equal(got[1], v) and np.array_equal(got[3], ev)
