"""A pool that is only dropped lives as long as a tensor views its memory."""
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_views_keep_a_dropped_pool_alive():
    import paged_kv_cache_227_gb300 as pa

    def views():
        pool = pa.Pool(512, 4, torch.bfloat16)
        pool.k.fill_(1.5)
        pool.v.fill_(-2.0)
        return pool.k, pool.v[3:5], pool._h

    k, v, handle = views()
    gc.collect()
    assert handle.ptr, "the views hold the pool"
    assert float(k.float().mean()) == 1.5 and float(v.float().mean()) == -2.0
    torch.cuda.synchronize()


def test_a_dropped_pool_without_views_is_released():
    import paged_kv_cache_227_gb300 as pa
    torch.cuda.synchronize()
    gc.collect()
    before = torch.cuda.mem_get_info()[0]
    pool = pa.Pool(65536, 8, torch.float16)     # 4 GiB
    assert torch.cuda.mem_get_info()[0] <= before - (4 << 30)
    del pool
    gc.collect()
    assert torch.cuda.mem_get_info()[0] > before - (1 << 30)


def test_close_releases_at_once_and_twice_is_fine():
    import paged_kv_cache_227_gb300 as pa
    pool = pa.Pool(16, 1, torch.float16)
    pool.close()
    assert not pool.handle and pool.k is None
    pool.close()
