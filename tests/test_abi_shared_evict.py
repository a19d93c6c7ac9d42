"""Refusals of the block eviction over shared pages, in the library and in the binding.  Nothing here launches a kernel."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_kvc_gb300 import build, kvc as k
    build.build()
    k.load()
    return k


@pytest.mark.parametrize("want,word,shares,n_blocks,recent", [
    (1, "null shares", None, 8, 1), (3, "aligned", 4098, 8, 1), (2, "n_blocks", 4096, 0, 1), (2, "n_blocks", 4096, -3, 1),
    (1, "recent_blocks", 4096, 8, 0)])
def test_library_refusals(kvc, want, word, shares, n_blocks, recent):
    pt = kvc.kvc_page_table()
    pt.table = pt.n_blocks = pt.len = pt.score = 4096
    pt.batch, pt.max_blocks = 2, 4
    fp = kvc.kvc_free_pool()
    fp.ids, fp.top, fp.capacity = 4096, 4096, 8
    st = kvc.load().kvc_block_accumulate_evict_shared(4096, 64, 4096, 4, 16, ctypes.byref(pt), ctypes.byref(fp), shares, n_blocks,
                                                      3, recent, None, None)
    assert st == want and word in kvc.kvc_last_error()


@pytest.mark.parametrize("shares", [torch.zeros(8, dtype=torch.int64), torch.zeros(16, dtype=torch.int32)[::2]])
def test_binding_refusals(kvc, shares):
    B, mb = 2, 4
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pt = kvc.page_table_view(i32(B, mb), i32(B), i32(B), torch.zeros(B, mb))
    free = kvc.free_pool_view(i32(8), i32(1))
    with pytest.raises(ValueError, match="shares"):
        kvc.kvc_block_accumulate_evict(torch.zeros(B, 4, mb * 16), torch.zeros(B, 4), pt, free, block_size=16, budget_blocks=3,
                                       recent_blocks=1, shares=shares)
