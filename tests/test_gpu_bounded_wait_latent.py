"""The bounded waits of the latent expansion.

A warp that waits for another without a limit turns a reported timeout into a kernel that never
ends, so its warps may meet only through waits that give up.  On the GPU,
KVC_TEST_STARVE makes the waits run out without any fault: nothing is copied, so nothing can be
landing in shared memory when a block exits.
"""
import os
import re
import time

import pytest
import torch

from gpu_helpers import cuda_or_skip, lib
from tree_ref import SENTINEL, randn

KVC_DEV_TIMEOUT = 7


def test_warps_meet_through_bounded_waits_only():
    """No named barrier, whose wait has no limit, hands work from one warp to another."""
    from kv_cache_compression_kvc_gb300 import build
    with open(os.path.join(build.CSRC, "latent_expand_tc.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"\bbar_sync\b|\bbar_arrive\b|\bbar_any\b|\bbar\.\w+", code)
    # one barrier over the block before the roles, two behind them
    assert len(re.findall(r"__syncthreads\(\)", code)) == 3


# one accumulator a head, two (d_head 256), two stages at least, a block of many tiles
@pytest.mark.gpu
@pytest.mark.parametrize("B,H,R,E,D,lens", [
    (1, 2, 128, 0, 64, [700]),
    (2, 32, 512, 64, 128, [4096, 4000]),
    (3, 5, 256, 32, 256, [1, 0, 1300]),
    (60, 3, 512, 64, 256, [900]),
])
def test_expand_wait_runs_out_and_next_call_is_exact(B, H, R, E, D, lens):
    dev = cuda_or_skip()
    kvc = lib()
    cap = max(lens)
    c = randn((B, cap, R + E), 1, dev, torch.bfloat16)
    wk, wv = randn((H, D - E, R), 2, dev, torch.bfloat16), randn((H, D, R), 3, dev, torch.bfloat16)
    ln = torch.tensor([lens[b % len(lens)] for b in range(B)], dtype=torch.int32, device=dev)

    def call(starve):
        k, v = (torch.full((B, H, cap, D), SENTINEL, dtype=torch.bfloat16, device=dev) for _ in range(2))
        cache = kvc.latent_cache_view(c, R)
        cache.reserved = kvc.KVC_TEST_STARVE if starve else 0
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        kvc.kvc_latent_expand(cache, wk, wv, kvc.cache_view(k, v), len=ln)
        code = kvc.kvc_device_status()
        return k, v, code, time.perf_counter() - t0

    k0, v0, code, _ = call(False)
    assert code == 0
    # every block gives up on its first wait and still finishes
    _, _, code, seconds = call(True)
    assert code == KVC_DEV_TIMEOUT and seconds < 10.0
    k1, v1, code, _ = call(False)
    assert code == 0 and torch.equal(k0, k1) and torch.equal(v0, v1)
