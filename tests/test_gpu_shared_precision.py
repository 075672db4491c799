"""The weights of a long prefix behind one token that takes most of it.

The scores are exact by construction (one nonzero dim, scale ln 2, whole
numbers), so what is left is the weights' own precision: with a weight p taken
relative to the largest, fp16 pools carry p to 2^-11 (16-bit output) or 2^-23
(fp32 output: half a step of what the first rounding left) of itself, and not
below 2^-32 absolute (half of fp16's least, 2^-25, of a weight times 2^7); bf16
to 2^-8 or 2^-17 of itself at any size.  The exponent is off by 32 * 2^-23 log2 units at
most, a relative 2^-18 with the unit's own 2^-22, and the sums of L terms by L *
2^-23 if every addition truncates."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, cuda, half_step, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


@pytest.mark.parametrize("tail", ["equal", "spread"])
@pytest.mark.parametrize("sink", [9, 14, 20, 23, 26, 28])
@pytest.mark.parametrize("out16", [False, True])
@pytest.mark.parametrize("members", [6, 40])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_tail_behind_a_sink(pa, dtype, members, out16, sink, tail):
    """So many groups (behind the same blocks) that most have their whole prefix
    in one CTA's range, against one running maximum."""
    P, ng, Hq, Hkv = 256, 100 if members == 6 else 60, 8, 2
    B, L = ng * members, P * BS + 1
    rng = np.random.default_rng(sink)
    perm = rng.permutation(P + B).astype(np.int32)
    tables = np.concatenate([np.tile(perm[:P], (B, 1)), perm[P:, None]], 1)
    # log2 weights of the prefix's tokens relative to the sink (token 0, value 0); the others' values are 1
    s = np.full((P, BS), -float(sink)) if tail == "equal" else -sink - rng.integers(0, 4, (P, BS)).astype(np.float64)
    s[0, 0] = 0
    pool = pa.Pool(P + B, Hkv, dtype)  # (zeros: the members' own tokens have score 0, value 0)
    at = torch.from_numpy(perm[:P].astype(np.int64)).cuda()
    pool.k[at, :, :, 0] = torch.from_numpy(s + sink).to(dtype).cuda()[:, None, :]
    v = torch.ones(P, BS, device="cuda")
    v[0, 0] = 0
    pool.v[at] = v.to(dtype)[:, None, :, None].expand(P, Hkv, BS, D)
    q = torch.zeros(B, Hq, D, dtype=dtype, device="cuda")
    q[:, :, 0] = 1.0
    out = torch.empty(B, Hq, D, dtype=dtype if out16 else torch.float32, device="cuda")
    pa.pa_decode_shared(pool, q, cuda(tables), cuda(np.full(B, L, np.int32)), float(np.log(2.0)), out,
                        cuda((members * np.arange(ng + 1)).astype(np.int32)), cuda(np.arange(B, dtype=np.int32)),
                        cuda(np.full(ng, P, np.int32)))
    ok(pa, pool)
    p = 2.0 ** s.reshape(-1)
    want = p[1:].sum() / (p.sum() + 2.0 ** -sink)
    if dtype == torch.float16:
        rel, floor = (2.0 ** -11 if out16 else 2.0 ** -23), 2.0 ** -32
    else:
        rel, floor = (2.0 ** -8 if out16 else 2.0 ** -17), 0.0
    tol = want * (rel + 2.0 ** -17 + L * 2.0 ** -23) + floor * L
    if out16:
        tol += half_step(dtype) * (want + tol) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    err = float((out.double() - want).abs().max())
    assert err <= tol, (err, tol, want)
    pool.close()
