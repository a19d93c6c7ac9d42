"""Pages whose keys of one head take 2^31 bytes: the calls that copy pages refuse them (a warp copies such a run and
counts its bytes in 32 bits; they would be left out without a word)."""
import ctypes

import pytest

from test_abi_pages_q8 import SHAPE, K, lib, stack, table  # noqa: F401

B_ = ctypes.byref


@pytest.mark.parametrize("dtype,eb", [(0, 4), (1, 2)])
@pytest.mark.parametrize("call", ["kvc_pages_reorder", "kvc_pages_compact"])
def test_pages_of_two_gigabytes_are_refused(lib, K, call, dtype, eb):  # noqa: F811
    pool = K.kvc_block_pool()
    pool.k = pool.v = 4096
    pool.dtype, pool.n_blocks, pool.n_heads_kv, pool.d_head = dtype, 8, 1, 256
    pool.block_size = 2 ** 31 // (256 * eb)
    args = (B_(pool), None, None, B_(table(K, max_blocks=2)), B_(stack(K)), 4096, None, 4096)
    assert getattr(lib, call)(*args, 4096, 1 << 30, None) == SHAPE and "2^31" in K.kvc_last_error()
    # a page that fits passes this check and fails the next one (no workspace)
    pool.block_size -= 256
    assert getattr(lib, call)(*args, None, 0, None) != SHAPE
