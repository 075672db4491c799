"""Host side of the 8-bit cache: refusals that need no GPU, and the tests' own
64-bit definitions against independent values."""
import ctypes
import types

import numpy as np
import pytest
import torch

import paged_kv_cache_227_gb300 as pa

from ._ops8 import E4M3, KINDS, TOP, decode8, encode8, need8, runs_of, type8, write8


def fake_pool(dtype, n_kv_heads=2):
    return types.SimpleNamespace(handle=None, dtype=dtype, n_kv_heads=n_kv_heads, device=torch.device("cuda", 0))


BF, I32, I64, F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


def test_host_tensors_are_refused():
    q, kv, w = torch.zeros(3, 4, 128, dtype=BF), torch.zeros(3, 2, 128, dtype=BF), torch.ones(128, dtype=BF)
    turn = (torch.zeros(1, 3, dtype=I32), torch.zeros(64, dtype=F32), [0] * 64, torch.zeros(3, dtype=I64), q)
    p8 = fake_pool(torch.int8)
    with pytest.raises(ValueError, match="must be on the GPU"):
        pa.pa_norm_rope_append(fake_pool(BF), q, kv, kv, w, w, *turn)
    with pytest.raises(ValueError, match="must be on the GPU"):
        pa.pa_norm_rope_append8(p8, q, kv, kv, w, w, *turn)
    with pytest.raises(ValueError, match="must be on the GPU"):
        pa.pa_cache_append8(p8, kv, kv, torch.zeros(3, dtype=I64))
    with pytest.raises(ValueError, match="must be on the GPU"):
        pa.pa_decode8(p8, q, torch.zeros(3, 2, dtype=I32), torch.zeros(3, dtype=I32), 0.1, q.float())
    with pytest.raises(ValueError, match="must be on the GPU"):
        pa.pa_copy_blocks8(p8, torch.zeros(3, dtype=I32), torch.zeros(3, dtype=I32))


def test_row_types_are_refused():
    p8 = fake_pool(torch.int8)
    f = torch.zeros(3, 4, 128)
    with pytest.raises(TypeError, match="fp16 or bf16"):
        pa.pa_decode8(p8, f, torch.zeros(3, 2, dtype=I32), torch.zeros(3, dtype=I32), 0.1, f)
    with pytest.raises(TypeError, match="fp16 or bf16"):
        pa.pa_cache_append8(p8, f, f, torch.zeros(3, dtype=I64))
    with pytest.raises(TypeError, match="torch.Tensor"):
        pa.pa_norm_rope_append8(p8, None, f, f, None, None, None, None, [0], None, None)
    with pytest.raises(TypeError, match="one Pool and one Pool8"):
        pa.pa_quantize_blocks(fake_pool(BF), torch.zeros(1, dtype=I32), p8, torch.zeros(1, dtype=I32))


def test_a_pool_of_the_other_kind_is_refused():
    """A pa_pool8_t is no pa_pool_t: neither call may reach the library with the other's handle."""
    p8 = pa.Pool8.__new__(pa.Pool8)
    with pytest.raises(TypeError, match="takes a Pool, got a Pool8"):
        p8.handle
    with pytest.raises(TypeError, match="takes a Pool, got a Pool8"):
        pa.pa_check(p8, types.SimpleNamespace(cuda_stream=0))
    for call in (pa.pa_check8, lambda p, s: pa.decode8_workspace_for(p, torch.zeros(1, 4, 128), torch.zeros(1, 1), s)):
        with pytest.raises(TypeError, match="takes a Pool8"):
            call(fake_pool(BF), types.SimpleNamespace(cuda_stream=0))


def test_null_pools_and_bad_sizes_are_refused():
    L, bad, none = pa.lib, pa.PA_ERR_INVALID, None
    turn = (none, 1, none, none, 128, 0, none, 1, none, 0, none)
    assert L.pa_norm_rope_append(none, none, 0, 1, none, 0, none, 0, none, none, 1e-6, *turn) == bad
    assert L.pa_norm_rope_append8(none, pa.PA_BF16, none, 0, 1, none, 0, none, 0, none, none, 1e-6, *turn) == bad
    assert L.pa_cache_append8(none, pa.PA_BF16, none, none, none, 1, none) == bad
    assert L.pa_decode8_workspace_bytes(none, 1, 1, 1) == 0
    assert L.pa_decode8(none, none, pa.PA_BF16, none, 1, none, 1, 8, 1.0, none, 2, none, 0, none) == bad
    assert L.pa_copy_blocks8(none, none, none, 1, none) == bad
    assert L.pa_quantize_blocks(none, none, none, none, none, 1, none) == bad
    assert L.pa_dequantize_blocks(none, none, none, none, 1, none) == bad
    assert L.pa_check8(none, none, none) == bad and L.pa_pool8_info(none, none, none) == bad
    assert L.pa_pool8_destroy(none) == pa.PA_OK
    h = ctypes.c_void_p()
    for n, bs, hk, d, t, want in ((0, 16, 2, 128, 3, bad), (4, 32, 2, 128, 3, pa.PA_ERR_UNSUPPORTED),
                                  (4, 16, 2, 64, 4, pa.PA_ERR_UNSUPPORTED), (4, 16, 2, 128, 1, pa.PA_ERR_UNSUPPORTED),
                                  (1 << 24, 16, 8, 128, 4, pa.PA_ERR_UNSUPPORTED)):
        assert L.pa_pool8_create(n, bs, hk, d, t, ctypes.byref(h)) == want
    assert L.pa_pool8_create(4, 16, 2, 128, 3, none) == bad


def test_pool8_bytes_are_half_of_a_16_bit_pool():
    for t in (pa.PA_E4M3, pa.PA_INT8):
        assert 2 * pa.lib.pa_pool8_bytes(7, 16, 5, 128, t) == pa.lib.pa_pool_bytes(7, 16, 5, 128, pa.PA_BF16)
    assert pa.lib.pa_pool8_bytes(7, 16, 5, 128, pa.PA_BF16) == 0 and pa.lib.pa_pool8_bytes(7, 8, 5, 128, pa.PA_INT8) == 0


def test_codes_of_the_definition():
    assert np.array_equal(E4M3, torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 4, 20000),
                        (E4M3[:126] + E4M3[1:127]) / 2])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(encode8(x, "e4m3"), want)
    for kind in KINDS:
        c = np.arange(256, dtype=np.uint8)
        v = decode8(c, kind)
        keep = np.isfinite(v) & (np.abs(v) <= TOP[kind])
        assert np.array_equal(encode8(v[keep], kind), c[keep])
    assert type8("int8") is torch.int8


@pytest.mark.parametrize("kind", KINDS)
def test_exponents_of_the_definition(kind):
    for x in (-126, -7, 0, 100):
        at = TOP[kind] * 2.0 ** x
        assert need8(at, kind) == x + 127
        assert need8(np.nextafter(at, np.inf), kind) == x + 128
    assert need8(0.0, kind) == 1 and need8(2.0 ** -149, kind) == 1
    assert need8(np.inf, kind) == 255 and need8(np.nan, kind) == 255


def test_runs_of_the_definition():
    assert runs_of([5, 6, 7, 20, 21, -1, 22, 14, 15, 16, 17, 99, 3], 64) == [[0, 1, 2], [3, 4], [6], [7, 8], [9, 10], [12]]


def test_write_of_the_definition_grows_and_restarts():
    codes, exps = np.zeros((2, 1, 16, 128), np.uint8), np.zeros((2, 1), np.uint8)
    row = lambda x: np.full((1, 1, 128), x, np.float64)  # noqa: E731
    codes, exps = write8(codes, exps, row(127.0), [0], "int8")
    assert exps[0, 0] == 127 and (codes[0, 0, 0] == 127).all()
    codes, exps = write8(codes, exps, row(5.0), [1], "int8")
    assert exps[0, 0] == 127 and (codes[0, 0, 1] == 5).all(), "a scale that holds the row stays"
    codes, exps = write8(codes, exps, row(300.0), [2], "int8")
    assert exps[0, 0] == 129 and codes[0, 0, :3, 0].tolist() == [32, 1, 75], "127 / 4 and 5 / 4 to nearest even"
    codes, exps = write8(codes, exps, row(1.0), [0], "int8")
    assert exps[0, 0] == need8(1.0, "int8") and codes[0, 0, :3, 0].tolist() == [64, 1, 75], "started afresh"
    codes, exps = write8(codes, exps, row(np.nan), [1], "int8")
    assert exps[0, 0] == 255
