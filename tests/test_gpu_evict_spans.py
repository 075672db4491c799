"""Eviction with every kernel of the selection: which one runs goes by the
width of the table, so each width is taken on both sides of its limits, with a
long and a short row in the same batch and all kinds of sums."""
import pytest
import torch

from .test_gpu_evict import BS, run_and_check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_227_gb300 as pa
    return pa


@pytest.mark.parametrize("place", ["in place", "fresh"])
@pytest.mark.parametrize("kind", ["ties", "equal", "odd"])
@pytest.mark.parametrize("span", [2048, 2064, 4096, 4112, 8192, 8208, 16384, 16400, 32768, 32784, 65536, 65552])
def test_both_sides_of_each_limit(pa, span, kind, place):
    long = span - 5
    run_and_check(pa, [long, 700], [long // 3, 77], 4, 33, 2, torch.bfloat16, kind, place, seed=span)
    # short rows in a wide table
    run_and_check(pa, [900], [500], 0, 1, 1, torch.float16, kind, place, seed=span + 1, extra_width=(span - 912) // BS)


@pytest.mark.parametrize("keep", [1, 64, 8192, 8193, 69999])
@pytest.mark.parametrize("kind", ["ties", "equal", "odd"])
def test_ties_across_the_tiles_of_a_long_row(pa, kind, keep):
    run_and_check(pa, [70000], [keep], 1, 7, 1, torch.float16, kind, "in place", seed=keep)
