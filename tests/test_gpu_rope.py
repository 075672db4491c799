"""Rotary append against its 64-bit definition.

Tolerance, from the arithmetic: the angle in turns is off by at most 2^-23 (two
32-bit roundings of values below 1) for |position| <= 2^24, and by 2^-19.5 for
any 32-bit position (the low part of the product, up to 10 turns, is rounded at
2^-24 relative, twice), so cos and sin are off by 2 pi times that and two units
of 2^-24 of their own; the two products and the sum add 3 * 2^-24.  In all
below 2^-19 (far: 2^-16) of |x| + |y|, before the one rounding to 16 bits."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, cuda, half_step, ok, rand16, rope64, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


def axes_of(rot, n_axes, style):
    if style == "runs":
        share = rot // 2 // n_axes
        return [min(f // max(1, share), n_axes - 1) for f in range(rot // 2)]
    return [f % n_axes for f in range(rot // 2)]  # dealt in turn


def check(got, ref, x, dtype, rot, interleaved, tol):
    mag = np.abs(x).copy()
    i = np.arange(rot // 2)
    i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    pair = np.abs(x[..., i0]) + np.abs(x[..., i1])
    mag[..., i0] = mag[..., i1] = pair
    mag[..., rot:] = 0
    slack = tol * mag
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134  # half a step of the subnormals
    bound = half_step(dtype) * (np.abs(ref) + slack) + slack + tiny * (mag > 0)
    bad = np.abs(got - ref) > bound
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - ref).max()))


CASES = [  # n, Hq, Hkv, dtype, rot, axes, deal, interleaved, fused, far
    (1, 32, 8, torch.bfloat16, 128, 3, "runs", False, True, 1 << 20),
    (2, 4, 4, torch.float16, 16, 1, "runs", False, False, 5),
    (64, 32, 8, torch.bfloat16, 128, 3, "turn", False, True, 1 << 24),
    (33, 12, 2, torch.float16, 64, 4, "turn", True, False, 4096),
    (17, 40, 40, torch.float16, 96, 2, "runs", True, True, 100000),
    (129, 7, 1, torch.bfloat16, 48, 3, "runs", False, True, 2048),
    (1531, 1, 1, torch.float16, 128, 2, "turn", True, True, 1 << 24),
]


@pytest.mark.parametrize("n,Hq,Hkv,dtype,rot,n_axes,deal,interleaved,fused,far", CASES)
def test_against_the_definition(pa, n, Hq, Hkv, dtype, rot, n_axes, deal, interleaved, fused, far):
    rng = np.random.default_rng(n * 131 + rot)
    nb = -(-n // BS) + 3
    pool = pa.Pool(nb, Hkv, dtype)
    k0, v0 = rand16(rng, dtype, nb, Hkv, BS, D), rand16(rng, dtype, nb, Hkv, BS, D)
    pool.k.copy_(k0); pool.v.copy_(v0)
    if fused:
        qkv = rand16(rng, dtype, n, Hq + 2 * Hkv, D).cuda()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (rand16(rng, dtype, n, h, D).cuda() for h in (Hq, Hkv, Hkv))
    pos = rng.integers(-far, far, (n_axes, n), dtype=np.int64).astype(np.int32)
    pos[0, 0] = 0
    inv = (10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)
    ax = axes_of(rot, n_axes, deal)
    slots = rng.permutation(nb * BS)[:n].astype(np.int64)
    slots[n // 2::7] = -1  # padding tokens keep out of the cache
    qo = torch.full((n, Hq, D), float("nan"), dtype=dtype, device="cuda")
    pa.pa_rope_append(pool, q, k, v, cuda(pos), cuda(inv), ax, cuda(slots), qo, interleaved=interleaved)
    ok(pa, pool)
    tol = 2.0 ** -19
    x = to64(q)
    check(to64(qo), rope64(x, pos, inv, ax, interleaved), x, dtype, rot, interleaved, tol)
    x = to64(k)
    ref = rope64(x, pos, inv, ax, interleaved)
    rows = to64(pool.k).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)
    at = slots >= 0
    check(rows[slots[at]], ref[at], x[at], dtype, rot, interleaved, tol)
    want_v = to64(v0).transpose(0, 2, 1, 3).reshape(-1, Hkv, D).copy()
    want_v[slots[at]] = to64(v)[at]
    assert np.array_equal(to64(pool.v).transpose(0, 2, 1, 3).reshape(-1, Hkv, D), want_v), "v moves bit for bit"
    rest = np.ones(nb * BS, bool)
    rest[slots[at]] = False
    assert np.array_equal(rows[rest], to64(k0).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[rest]), "other slots untouched"
    pool.close()


def test_farthest_positions_and_zero_angle(pa):
    """Positions at the ends of 32 bits; position 0 returns the row's bits."""
    dtype, n = torch.float16, 6
    rng = np.random.default_rng(5)
    pool = pa.Pool(2, 1, dtype)
    q, k, v = (rand16(rng, dtype, n, 1, D).cuda() for _ in range(3))
    pos = np.array([[0, 2**31 - 1, -2**31, 2**24 + 1, 1 << 30, -1]], np.int32)
    inv = (500000.0 ** (-np.arange(0, 128, 2) / 128)).astype(np.float32)
    qo = torch.empty(n, 1, D, dtype=dtype, device="cuda")
    pa.pa_rope_append(pool, q, k, v, cuda(pos), cuda(inv), [0] * 64, torch.full((n,), -1, dtype=torch.int64, device="cuda"),
                      qo)
    ok(pa, pool)
    assert torch.equal(qo[0], q[0])
    x = to64(q)
    check(to64(qo), rope64(x, pos, inv, [0] * 64, False), x, dtype, 128, False, 2.0 ** -16)
    pool.close()


def test_in_place_other_stream_and_graph(pa):
    """q turned in place gives the bits of q_out apart; a captured call replays on new inputs."""
    dtype, n, Hq, Hkv = torch.bfloat16, 37, 8, 2
    rng = np.random.default_rng(6)
    pool = pa.Pool(8, Hkv, dtype)
    q, k, v = (rand16(rng, dtype, n, h, D).cuda() for h in (Hq, Hkv, Hkv))
    pos = cuda(rng.integers(0, 9000, (2, n)).astype(np.int32))
    inv = cuda((10000.0 ** (-np.arange(0, 128, 2) / 128)).astype(np.float32))
    ax = [f % 2 for f in range(64)]
    slots = cuda(rng.permutation(8 * BS)[:n].astype(np.int64))
    apart, inplace = torch.empty_like(q), q.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pa.pa_rope_append(pool, q, k, v, pos, inv, ax, slots, apart, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    kept = pool.k.clone()
    pa.pa_rope_append(pool, inplace, k, v, pos, inv, ax, slots, inplace)
    assert torch.equal(apart, inplace) and torch.equal(kept, pool.k)
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(q)
    with torch.cuda.graph(g):
        pa.pa_rope_append(pool, q, k, v, pos, inv, ax, slots, out)
    q2 = rand16(rng, dtype, n, Hq, D).cuda()
    q.copy_(q2)
    g.replay()
    pa.pa_rope_append(pool, q2, k, v, pos, inv, ax, slots, apart)
    assert torch.equal(out, apart)
    ok(pa, pool)
    pool.close()


def test_bad_slots_are_reported_and_skipped(pa):
    dtype, n = torch.bfloat16, 3
    pool = pa.Pool(2, 1, dtype)
    q, k, v = (torch.ones(n, 1, D, dtype=dtype, device="cuda") for _ in range(3))
    pos = torch.zeros(1, n, dtype=torch.int32, device="cuda")
    inv = torch.ones(8, dtype=torch.float32, device="cuda")
    qo = torch.zeros_like(q)
    slots = torch.tensor([1, 32, -5], dtype=torch.int64, device="cuda")
    pa.pa_rope_append(pool, q, k, v, pos, inv, [0] * 8, slots, qo)
    assert pa.pa_check(pool) == (pa.PA_ERR_DEVICE_CHECK, 32)
    assert torch.equal(qo, q), "q is turned whatever the slot"
    assert float(pool.k.float().sum()) == D and float(pool.v.float().sum()) == D
    pool.close()


def test_refusals(pa):
    dtype = torch.bfloat16
    pool = pa.Pool(2, 2, dtype)
    z = lambda *s, t=dtype: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    good = dict(q=z(3, 4, D), k_new=z(3, 2, D), v_new=z(3, 2, D), positions=z(2, 3, t=torch.int32),
                inv_freq=z(64, t=torch.float32), axis_of_pair=[0] * 64, slot_mapping=z(3, t=torch.int64), q_out=z(3, 4, D))
    pa.pa_rope_append(pool, **good)
    for change, error in [
            (dict(axis_of_pair=[2] * 64), pa.PagedAttentionError),      # past the axes
            (dict(axis_of_pair=[-1] * 64), ValueError),
            (dict(inv_freq=z(63, t=torch.float32)), ValueError),
            (dict(inv_freq=z(4, t=torch.float32), axis_of_pair=[0] * 4), pa.PagedAttentionError),   # rot_dim 8
            (dict(inv_freq=z(72, t=torch.float32), axis_of_pair=[0] * 72), pa.PagedAttentionError),  # rot_dim 144
            (dict(inv_freq=z(0, t=torch.float32), axis_of_pair=[]), pa.PagedAttentionError),
            (dict(positions=z(5, 3, t=torch.int32)), pa.PagedAttentionError),
            (dict(positions=z(2, 4, t=torch.int32)), ValueError),
            (dict(q=z(3, 4, D, t=torch.float16)), TypeError),
            (dict(k_new=z(3, 4, D)), ValueError),
            (dict(q=z(3, D, 4).transpose(1, 2)), ValueError),           # heads not contiguous
            (dict(q=z(3, 4 * D + 4)[:, :4 * D].view(3, 4, D)), pa.PagedAttentionError),   # token stride not of 8
            (dict(q=z(1, 4, D).expand(3, 4, D), q_out=z(3, 4, D)), pa.PagedAttentionError),  # stride 0
            (dict(q=z(3 * 4 * D + 4)[4:].view(3, 4, D)), pa.PagedAttentionError),          # 8-byte aligned only
            (dict(slot_mapping=z(3, t=torch.int32)), TypeError)]:
        with pytest.raises(error):
            pa.pa_rope_append(pool, **{**good, **change})
    qo = z(3, 5, D)
    with pytest.raises(pa.PagedAttentionError):  # in place with another stride
        pa.pa_rope_append(pool, **{**good, "q": qo[:, :4].view(3, 4, D), "q_out": qo.view(-1)[:3 * 4 * D].view(3, 4, D)})
    none = dict(good, q=z(0, 4, D), k_new=z(0, 2, D), v_new=z(0, 2, D), positions=z(2, 0, t=torch.int32),
                slot_mapping=z(0, t=torch.int64), q_out=z(0, 4, D))
    pa.pa_rope_append(pool, **none)
    ok(pa, pool)
    pool.close()
