"""What the cache operators' binding makes of host-side arguments.  A stand-in
pool on the CPU with a null handle: arguments that pass the binding's checks
reach the library, which refuses the pool."""
import types

import numpy as np
import pytest
import torch

import paged_kv_cache_227_gb300 as pa

POOL = types.SimpleNamespace(handle=None, dtype=torch.bfloat16, n_kv_heads=2, device=torch.device("cpu"))
STREAM = types.SimpleNamespace(cuda_stream=0)


def rope(axis_of_pair, pairs=64, n=3):
    q, kv = torch.zeros(n, 4, 128, dtype=torch.bfloat16), torch.zeros(n, 2, 128, dtype=torch.bfloat16)
    pa.pa_rope_append(POOL, q, kv, kv, torch.zeros(2, n, dtype=torch.int32), torch.zeros(pairs), axis_of_pair,
                      torch.zeros(n, dtype=torch.int64), q, stream=STREAM)


@pytest.mark.parametrize("axes", [[0, 1] * 32, (0, 1) * 32, bytes(64), bytearray(64), np.arange(64) % 2,
                                  (np.arange(64) % 2).astype(np.int32), np.zeros(64, np.uint8), torch.arange(64) % 2,
                                  (f % 2 for f in range(64))])
def test_axes_as_any_sequence_of_ints(axes):
    with pytest.raises(pa.PagedAttentionError):  # (the null pool)
        rope(axes)


def test_axes_that_are_none_are_refused():
    for axes, error in [(64, TypeError), (np.zeros(64), TypeError), ([0.5] * 64, TypeError), (np.full(64, 256), ValueError),
                        (np.full(64, -1), ValueError), (np.zeros(8, np.int64), ValueError), (None, TypeError)]:
        with pytest.raises(error):
            rope(axes)


def test_tables_too_wide_to_be_walked_in_32_bits_are_refused():
    """Steps of a walk go past a row's end by less than 2^20 positions.  (The pool
    is a block of memory that claims a device which is never the current one:
    what is not refused for its size is refused for that.)"""
    import ctypes
    room = (ctypes.c_char * 1024)()
    at = (ctypes.addressof(room) + 63) // 64 * 64
    ints = (ctypes.c_int * 4).from_address(at + 128)  # behind the 128-byte tensor map
    ints[0], ints[1], ints[2], ints[3] = 4, 1, pa.PA_BF16, -7
    widest = (1 << 27) - (1 << 16)

    def evict(w, wd):
        return pa.lib.pa_evict(at, 256, 256, 256, w, 256 if wd else None, wd, 256, 256, 1, 0, 0, 512, 256, None)

    assert evict(widest, 0) == evict(widest, widest) == pa.PA_ERR_INVALID
    assert evict(widest + 1, 0) == evict(4, widest + 1) == evict((1 << 27) - 1, 0) == pa.PA_ERR_UNSUPPORTED

    def weights(w):
        return pa.lib.pa_decode_weights(at, 256, 256, w, 256, 1, 1, 1.0, 256, pa.PA_BF16, 256, 1.0, 256, 1 << 62, None)

    assert weights(widest) == pa.PA_ERR_INVALID
    assert weights(widest + 1) == weights((1 << 27) - 1) == pa.PA_ERR_UNSUPPORTED
