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
