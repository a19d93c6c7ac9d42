"""GPU: the bounded waits of the draft-tree and latent attention, made to run out without any fault.

With KVC_TEST_STARVE nothing is loaded, so the first waits of every block give up after a short bounded
spin.  The call must finish and report KVC_DEV_TIMEOUT, and the next one must give the same bits as
before; no copy is ever issued in this mode, so none can be landing when a block exits.
"""
import time

import pytest
import torch

from gpu_helpers import cuda_or_skip, lib
from tree_ref import randn, tree_masks

pytestmark = pytest.mark.gpu
KVC_DEV_TIMEOUT = 7
BF16 = torch.bfloat16


def check(kvc, call, draft):
    """call(out, lse) before, during and after a starved one."""
    out0, lse0 = call()
    assert kvc.kvc_device_status() == 0
    draft.reserved = kvc.KVC_TEST_STARVE
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call()
    assert kvc.kvc_device_status() == KVC_DEV_TIMEOUT
    assert time.perf_counter() - t0 < 10.0
    draft.reserved = 0
    out1, lse1 = call()
    assert kvc.kvc_device_status() == 0
    assert torch.equal(out0, out1) and torch.equal(lse0, lse1)
    assert bool(torch.isfinite(out1).all())


# (Hkv, G, D, T, lens of the rows): 64 and 128 rows a tile, the weights through shared and through tensor
# memory, whole and split pairs, several row tiles, changes of pair inside a block
@pytest.mark.parametrize("B,Hkv,G,D,T,lens", [
    (1, 1, 2, 64, 4, [100]),
    (1, 2, 4, 64, 40, [5000, 3000]),
    (2, 2, 4, 128, 16, [20000, 0, 129, 7000]),
    (2, 2, 4, 128, 64, [20000, 1, 129, 7000]),
    (40, 8, 1, 128, 8, [817, 5, 0]),
    (2, 2, 6, 256, 11, [5000, 64]),
    (1, 1, 2, 256, 5, [700]),
])
def test_tree_wait_runs_out_and_next_call_is_exact(B, Hkv, G, D, T, lens):
    dev = cuda_or_skip()
    kvc = lib()
    cap = max(lens)
    q = randn((B, T, Hkv * G, D), 1, dev, BF16)
    k, v = randn((B, Hkv, cap, D), 2, dev, BF16), randn((B, Hkv, cap, D), 3, dev, BF16)
    kd, vd = randn((B, T, Hkv, D), 4, dev, BF16), randn((B, T, Hkv, D), 5, dev, BF16)
    ln = torch.tensor([lens[i % len(lens)] for i in range(B * Hkv)], dtype=torch.int32, device=dev)
    draft, cache = kvc.make_draft(kd, vd, mask=tree_masks(B, T, 6).to(dev)), kvc.cache_view(k, v)
    ws = kvc.tree_workspace(B, Hkv * G, Hkv, D, T, BF16, dev)

    def call():
        lse = torch.empty(q.shape[:3], device=dev)
        return kvc.kvc_decode_attn_tree(q, cache, draft, scale=D ** -0.5, len=ln, lse=lse, ws=ws), lse

    check(kvc, call, draft)


@pytest.mark.parametrize("bs", [8, 32, 256])
def test_paged_wait_runs_out_and_next_call_is_exact(bs):
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv, G, D, T, n = 5, 3, 2, 128, 7, 1500
    mb = -(-n // bs)
    kp, vp = randn((Hkv, B * mb, bs, D), 1, dev, BF16), randn((Hkv, B * mb, bs, D), 2, dev, BF16)
    table = torch.arange(B * mb, dtype=torch.int32, device=dev).flip(0).view(B, mb).contiguous()
    ln = torch.tensor([n, 3, 700, 0, 129], dtype=torch.int32, device=dev)
    nb = (ln + bs - 1) // bs
    pool = kvc.block_pool_view(kp, vp)
    pt = kvc.page_table_view(table, nb.to(torch.int32), ln, torch.zeros((B, mb), device=dev))
    q = randn((B, T, Hkv * G, D), 3, dev, BF16)
    draft = kvc.make_draft(randn((B, T, Hkv, D), 4, dev, BF16), randn((B, T, Hkv, D), 5, dev, BF16))

    def call():
        lse = torch.empty(q.shape[:3], device=dev)
        return kvc.kvc_decode_attn_tree_paged(q, pool, pt, draft, scale=0.1, lse=lse), lse

    check(kvc, call, draft)


@pytest.mark.parametrize("B,H,R,E,T,lens", [
    (1, 16, 512, 64, 1, [1000]),
    (7, 16, 512, 64, 2, [8000, 3, 0, 640]),
    (2, 128, 512, 64, 4, [3000, 70]),
    (3, 24, 256, 0, 3, [500, 2000]),
    (2, 8, 128, 32, 16, [129]),
])
def test_latent_wait_runs_out_and_next_call_is_exact(B, H, R, E, T, lens):
    dev = cuda_or_skip()
    kvc = lib()
    q, c = randn((B, T, H, R + E), 1, dev, BF16), randn((B, max(lens), R + E), 2, dev, BF16)
    ln = torch.tensor([lens[b % len(lens)] for b in range(B)], dtype=torch.int32, device=dev)
    draft = kvc.make_draft(randn((B, T, R + E), 3, dev, BF16))
    cache = kvc.latent_cache_view(c, R)

    def call():
        lse = torch.empty(q.shape[:3], device=dev)
        return kvc.kvc_decode_attn_latent(q, cache, draft, scale=0.05, len=ln, lse=lse), lse

    check(kvc, call, draft)
