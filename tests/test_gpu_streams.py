"""GPU: calls on another stream than the current one, without a workspace of the caller's: nothing that
the current stream allocates meanwhile shares memory with what the kernels use."""
import pytest
import torch

from gpu_helpers import cuda_or_skip, lib
from tree_ref import randn, tree_masks

pytestmark = pytest.mark.gpu


def cases(kvc, dev):
    B, Hkv, G, D, T, cap, bs = 2, 2, 4, 128, 12, 3000, 32
    bf = torch.bfloat16
    q, q1 = randn((B, T, Hkv * G, D), 1, dev, bf), randn((B, Hkv * G, D), 2, dev, bf)
    k, v = randn((B, Hkv, cap, D), 3, dev, bf), randn((B, Hkv, cap, D), 4, dev, bf)
    kd, vd = randn((B, T, Hkv, D), 5, dev, bf), randn((B, T, Hkv, D), 6, dev, bf)
    mask = tree_masks(B, T, 1).to(dev)
    draft, cache = kvc.make_draft(kd, vd, mask=mask), kvc.cache_view(k, v)
    mb = 90
    kp, vp = randn((Hkv, B * mb, bs, D), 7, dev, bf), randn((Hkv, B * mb, bs, D), 8, dev, bf)
    table = torch.randperm(B * mb, generator=torch.Generator().manual_seed(1)).view(B, mb).to(torch.int32).to(dev)
    ln = torch.full((B,), mb * bs - 5, dtype=torch.int32, device=dev)
    nb = torch.full((B,), mb, dtype=torch.int32, device=dev)
    pool, pt = kvc.block_pool_view(kp, vp), kvc.page_table_view(table, nb, ln, torch.zeros((B, mb), device=dev))
    c, cd = randn((B, cap, 576), 9, dev, bf), randn((B, T, 576), 10, dev, bf)
    ql = randn((B, T, 16, 576), 11, dev, bf)
    lat, ldraft = kvc.latent_cache_view(c, 512), kvc.make_draft(cd, mask=mask)
    return {
        "tree": lambda s: kvc.kvc_decode_attn_tree(q, cache, draft, scale=0.1, n_valid=cap, stream=s),
        "paged": lambda s: kvc.kvc_decode_attn_tree_paged(q, pool, pt, draft, scale=0.1, stream=s),
        "latent": lambda s: kvc.kvc_decode_attn_latent(ql, lat, ldraft, scale=0.05, n_valid=cap, stream=s),
        "decode": lambda s: kvc.kvc_decode_attn(q1, k, v, scale=0.1, n_valid=cap, stream=s),
    }


@pytest.mark.parametrize("name", ["tree", "paged", "latent", "decode"])
def test_temporaries_of_a_call_on_another_stream(name):
    dev = cuda_or_skip()
    kvc = lib()
    call = cases(kvc, dev)[name]
    want = call(None).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)          # the kernels start after what follows has been queued
    got = call(side)
    fills = [torch.full((n,), 0x5a, dtype=torch.uint8, device=dev)
             for n in [2 ** i for i in range(9, 25)] for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool((x == 0x5a).all()) for x in fills)
    assert torch.equal(got, want) and kvc.kvc_device_status() == 0
