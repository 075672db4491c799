"""Norms with the rotary append, into 16 bits, against the 64-bit definition.

Tolerance, from the arithmetic: the sum of squares has 128 terms of one sign in
chains of 8, then 4 additions: off by at most 12 * 2^-24 of itself, its inverse
root by half of that and 2^-22 (rsqrtf: 2 ulp); the two products add 2^-23.  In
all below 2^-20 of the normed value.  The rotation adds 2^-19 of |x| + |y|
(tests of the rotary append): 2^-18 of |x| + |y| of the normed pair covers both,
before the one rounding to 16 bits."""
import numpy as np
import pytest
import torch

from ._ops import BS, D, cuda, half_step, ok, rand16, to64
from ._ops8 import norm64, norm_rope64, rand_rows

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


def weight(rng, dtype):
    return torch.from_numpy(1 + 0.3 * rng.standard_normal(D).astype(np.float32)).to(dtype).cuda()


def pair_size(x, rot, interleaved):
    mag = np.abs(x).copy()
    i = np.arange(rot // 2)
    i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    mag[..., i0] = mag[..., i1] = np.abs(x[..., i0]) + np.abs(x[..., i1])
    return mag


def check(got, ref, normed, dtype, rot, interleaved):
    slack = 2.0 ** -18 * pair_size(normed, rot, interleaved)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134
    bad = np.abs(got - ref) > half_step(dtype) * (np.abs(ref) + slack) + slack + tiny
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - ref)[bad].max()))


class Tokens:
    def __init__(self, rng, n, Hq, Hkv, dtype, rot, n_axes, interleaved, fused=False, size=1.0):
        if fused:
            qkv = (rand_rows(rng, torch.float32, n, Hq + 2 * Hkv) * size).to(dtype)
            self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            self.q, self.k, self.v = ((rand_rows(rng, torch.float32, n, h) * size).to(dtype) for h in (Hq, Hkv, Hkv))
        self.pos = rng.integers(0, 5000, (n_axes, n)).astype(np.int32)
        self.inv = (10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)
        self.axes = [f % n_axes for f in range(rot // 2)]
        self.interleaved, self.rot, self.dtype = interleaved, rot, dtype
        self.q_out = torch.full((n, Hq, D), float("nan"), dtype=dtype, device="cuda")

    def want(self, x, w, eps=EPS):
        w = None if w is None else to64(w)
        x = to64(x)
        return norm_rope64(x, w, eps, self.pos, self.inv, self.axes, self.interleaved), norm64(x, w, eps)

    def args(self, wq, wk, slots):
        return (self.q, self.k, self.v, wq, wk, cuda(self.pos), cuda(self.inv), self.axes, cuda(np.asarray(slots, np.int64)),
                self.q_out)


CASES = [  # n, Hq, Hkv, dtype, rot, axes, interleaved, fused, norms
    (1, 32, 8, torch.bfloat16, 128, 1, False, True, "qk"),
    (3, 4, 4, torch.float16, 16, 1, False, False, "q"),
    (64, 32, 8, torch.bfloat16, 128, 3, True, True, "qk"),
    (33, 12, 2, torch.float16, 64, 2, True, False, "k"),
    (129, 7, 1, torch.bfloat16, 96, 1, False, True, "qk"),
    (1531, 5, 1, torch.float16, 128, 4, False, False, "qk"),
    # rows that wait in shared memory: query rows alone in a quad and not, a last quad with one row
    (420, 32, 8, torch.bfloat16, 128, 2, False, True, "qk"),
    (620, 30, 3, torch.float16, 64, 1, True, False, "qk"),
    (560, 27, 7, torch.bfloat16, 96, 1, False, True, "q"),
    (700, 40, 40, torch.float16, 128, 1, True, True, "k"),
]


@pytest.mark.parametrize("n,Hq,Hkv,dtype,rot,n_axes,interleaved,fused,norms", CASES)
def test_against_the_definition(pa, n, Hq, Hkv, dtype, rot, n_axes, interleaved, fused, norms):
    rng = np.random.default_rng(n * 7 + rot)
    nb = -(-n // BS) + 2
    pool = pa.Pool(nb, Hkv, dtype)
    k0 = rand16(rng, dtype, nb, Hkv, BS, D)
    pool.k.copy_(k0)
    t = Tokens(rng, n, Hq, Hkv, dtype, rot, n_axes, interleaved, fused)
    wq, wk = (weight(rng, dtype) if x in norms else None for x in "qk")
    slots = rng.permutation(nb * BS)[:n].astype(np.int64)
    slots[n // 2::5] = -1
    pa.pa_norm_rope_append(pool, *t.args(wq, wk, slots), eps=EPS, interleaved=interleaved)
    ok(pa, pool)
    ref, normed = t.want(t.q, wq)
    check(to64(t.q_out), ref, normed, dtype, rot, interleaved)
    at = slots >= 0
    ref, normed = t.want(t.k, wk)
    rows = to64(pool.k).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)
    check(rows[slots[at]], ref[at], normed[at], dtype, rot, interleaved)
    vrows = to64(pool.v).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)
    assert np.array_equal(vrows[slots[at]], to64(t.v)[at]), "v moves bit for bit"
    rest = np.setdiff1d(np.arange(nb * BS), slots[at])
    assert np.array_equal(rows[rest], to64(k0).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[rest])
    pool.close()


@pytest.mark.parametrize("far", [1 << 24, 1 << 31])
@pytest.mark.parametrize("n", [70, 700])
def test_far_positions(pa, n, far):
    """The angle in turns is off by 2^-23 up to 2^24 and by 2^-19.5 for any 32-bit position (tests of the
    rotary append): 2^-18 and 2^-16 of |x| + |y| with the norm's share, before the rounding."""
    rng = np.random.default_rng(far % 1000 + n)
    dtype = torch.float16
    t = Tokens(rng, n, 32, 2, dtype, 128, 2, False)
    t.pos = rng.integers(-far, far, (2, n), dtype=np.int64).astype(np.int32)
    pool, w = pa.Pool(-(-n // BS), 2, dtype), weight(rng, dtype)
    pa.pa_norm_rope_append(pool, *t.args(w, w, np.arange(n)))
    ref, normed = t.want(t.q, w)
    slack = (2.0 ** -18 if far <= 1 << 24 else 2.0 ** -16) * pair_size(normed, 128, False)
    assert (np.abs(to64(t.q_out) - ref) <= half_step(dtype) * (np.abs(ref) + slack) + slack + 2.0 ** -25).all()
    pool.close()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_no_weights_is_the_rotary_append_bit_for_bit(pa, dtype):
    rng = np.random.default_rng(5)
    t = Tokens(rng, 50, 6, 3, dtype, 64, 2, False)
    a, b = pa.Pool(6, 3, dtype), pa.Pool(6, 3, dtype)
    slots = rng.permutation(96)[:50]
    args = t.args(None, None, slots)
    pa.pa_norm_rope_append(a, *args)
    first = t.q_out.clone()
    pa.pa_rope_append(b, *args[:3], *args[5:])
    assert torch.equal(first, t.q_out) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


def test_a_normed_row_keeps_its_other_rows_apart(pa):
    """A row of zeros, of NaN and of infinities: only its own output shows it."""
    rng = np.random.default_rng(6)
    dtype = torch.bfloat16
    t = Tokens(rng, 9, 8, 2, dtype, 128, 1, False)
    clean = pa.Pool(2, 2, dtype)
    w = weight(rng, dtype)
    pa.pa_norm_rope_append(clean, *t.args(w, w, np.arange(9)))
    q_clean = t.q_out.clone()
    t.q[2, 3], t.q[4, 1, 7], t.q[5, 0, 100] = 0.0, float("nan"), float("inf")
    t.k[6, 1, 3] = float("nan")
    pool = pa.Pool(2, 2, dtype)
    pa.pa_norm_rope_append(pool, *t.args(w, w, np.arange(9)))
    assert (t.q_out[2, 3] == 0).all(), "zeros with eps stay zeros"
    assert torch.isnan(t.q_out[4, 1]).all() and torch.isnan(t.q_out[5, 0]).any()
    for i, h in ((2, 3), (4, 1), (5, 0)):
        t.q_out[i, h] = q_clean[i, h]
    assert torch.equal(t.q_out, q_clean)
    assert torch.isnan(pool.k[0, 1, 6]).all()
    pool.k[0, 1, 6] = clean.k[0, 1, 6]
    assert torch.equal(pool.k, clean.k) and torch.equal(pool.v, clean.v)


def test_in_place_streams_and_graphs(pa):
    rng = np.random.default_rng(7)
    dtype = torch.float16
    t = Tokens(rng, 40, 12, 2, dtype, 128, 1, True, fused=True)
    w = weight(rng, dtype)
    slots = rng.permutation(64)[:40]
    want = pa.Pool(4, 2, dtype)
    args = t.args(w, w, slots)
    pa.pa_norm_rope_append(want, *args, interleaved=True)
    q_want = t.q_out.clone()
    pool = pa.Pool(4, 2, dtype)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    pa.pa_norm_rope_append(pool, *args, interleaved=True, stream=st)
    st.synchronize()
    assert torch.equal(pool.k, want.k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_norm_rope_append(pool, *args, interleaved=True)
    pool.k.zero_(), t.q_out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(pool.k, want.k) and torch.equal(t.q_out, q_want)
    pa.pa_norm_rope_append(pool, t.q, *args[1:-1], t.q, interleaved=True)
    assert torch.equal(t.q, q_want), "q_out may be q"


def test_refusals(pa):
    rng = np.random.default_rng(8)
    dtype = torch.bfloat16
    pool = pa.Pool(2, 2, dtype)
    t = Tokens(rng, 5, 4, 2, dtype, 128, 1, False)
    w = weight(rng, dtype)
    for bad in (-1.0, float("nan"), float("inf")):
        with pytest.raises(pa.PagedAttentionError):
            pa.pa_norm_rope_append(pool, *t.args(w, w, range(5)), eps=bad)
    with pytest.raises(ValueError, match=r"q_weight must be \[128\]"):
        pa.pa_norm_rope_append(pool, *t.args(w[:64], w, range(5)))
    with pytest.raises(TypeError):
        pa.pa_norm_rope_append(pool, *t.args(w, w.float(), range(5)))
    with pytest.raises(pa.PagedAttentionError):  # not 16-byte aligned
        pa.pa_norm_rope_append(pool, *t.args(torch.zeros(129, dtype=dtype, device="cuda")[1:], w, range(5)))
    with pytest.raises(TypeError):
        pa.pa_norm_rope_append(pool, t.q.half(), *t.args(w, w, range(5))[1:])
    assert torch.isnan(t.q_out).all() and not pool.k.any(), "nothing was launched"
