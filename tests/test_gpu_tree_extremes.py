"""GPU: draft-tree and latent calls at the ends of their ranges: thousands of short pairs, the most
rows a pair can have, sequences that share one cache (a stride of zero)."""
import math

import pytest
import torch

from gpu_helpers import cuda_or_skip, lib
from tree_ref import SENTINEL, compare, randn, tolerance, tree_masks

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]


def reference(q, k, v, kd, vd, mask, lens, count, scale):
    """All pairs at once in 64 bits: q [B, T, Hq, Dk], k/v [B, H, S, .], kd/vd [B, T, H, .], lens
    [B, H], count [B].  Returns out, lse and the bounds on their errors."""
    B, T, Hq, Dk = q.shape
    H, S = k.shape[1], k.shape[2]
    G = Hq // H
    dt = q.dtype
    rows = q.double().view(B, T, H, G, Dk)
    keys = torch.cat([k.double(), kd.double().transpose(1, 2)], 2)
    values = torch.cat([v.double(), vd.double().transpose(1, 2)], 2)
    s = torch.einsum("bthgd,bhjd->bthgj", rows, keys) * scale
    mag = abs(scale) * torch.einsum("bthgd,bhjd->bthgj", rows.abs(), keys.abs())
    i = torch.arange(T, device=q.device)
    see = torch.arange(S, device=q.device) < lens[..., None]                     # [B, H, S]
    bits = ((mask[:, :, None] >> i) & 1 != 0) & (i < count[:, None])[:, None]    # [B, T, T]
    live = torch.cat([see[:, None].expand(B, T, H, S), bits[:, :, None].expand(B, T, H, T)], 3)[:, :, :, None]
    s = s.masked_fill(~live, -math.inf)
    lse = torch.logsumexp(s, dim=4)
    p = torch.exp(s - lse.masked_fill(lse == -math.inf, 0)[..., None])
    out = torch.einsum("bthgj,bhjd->bthgd", p, values)
    pv = torch.einsum("bthgj,bhjd->bthgd", p, values.abs())
    t_out, t_lse = tolerance(dt, Dk, S + T, pv, mag.masked_fill(~live, 0).amax(4), out, lse)
    return [x.reshape(B, T, Hq, *x.shape[4:]) for x in (out, lse, t_out, t_lse)]


def check(out, lse, q, k, v, kd, vd, mask, lens, count, scale, what):
    T = q.shape[1]
    o, z, t_out, t_lse = reference(q, k, v, kd, vd, mask, lens, count, scale)
    live = torch.arange(T, device=q.device) < count[:, None]
    assert bool((out[~live] == SENTINEL).all()) and bool((lse[~live] == SENTINEL).all()), what
    compare(out[live], o[live], t_out[live], f"{what} out")
    compare(lse[live], z[live], t_lse[live], f"{what} lse")


def lengths(shape, cap, seed, dev):
    gen = torch.Generator().manual_seed(seed)
    n = torch.randint(0, cap + 1, shape, generator=gen)
    n[torch.rand(shape, generator=gen) < 0.3] = 0
    return n.to(torch.int32).to(dev)


def counts(B, T, seed, dev):
    gen = torch.Generator().manual_seed(seed)
    n = torch.randint(0, T + 1, (B,), generator=gen)
    n[0] = T
    return n.to(torch.int32).to(dev)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,H,G,D,T,cap", [(2048, 4, 2, 64, 3, 40), (1031, 5, 1, 128, 2, 33),
                                           (600, 8, 20, 64, 4, 70), (520, 3, 2, 256, 2, 2000)])
def test_thousands_of_ragged_pairs(dtype, B, H, G, D, T, cap):
    """More pairs than lanes and blocks, a third of them empty: ranges of whole pairs and split ones."""
    dev = cuda_or_skip()
    kvc = lib()
    if cap > 1000:
        B //= 8
    q = randn((B, T, H * G, D), 1, dev, dtype)
    k, v = randn((B, H, cap, D), 2, dev, dtype), randn((B, H, cap, D), 3, dev, dtype)
    kd, vd = randn((B, T, H, D), 4, dev, dtype), randn((B, T, H, D), 5, dev, dtype)
    mask, lens, count = tree_masks(B, T, 6).to(dev), lengths((B, H), cap, 7, dev), counts(B, T, 8, dev)
    out, lse = torch.full_like(q, SENTINEL), torch.full(q.shape[:3], SENTINEL, device=dev)
    kvc.kvc_decode_attn_tree(q, kvc.cache_view(k, v), kvc.make_draft(kd, vd, mask=mask, count=count),
                             scale=D ** -0.5, len=lens, out=out, lse=lse)
    assert kvc.kvc_device_status() == 0
    check(out, lse, q, k, v, kd, vd, mask, lens, count, D ** -0.5, "pairs")


@pytest.mark.parametrize("dtype", TYPES)
def test_thousands_of_paged_sequences(dtype):
    dev = cuda_or_skip()
    kvc = lib()
    B, H, G, D, T, bs, mb = 1500, 3, 2, 64, 3, 16, 4
    kp, vp = randn((H, B * mb, bs, D), 1, dev, dtype), randn((H, B * mb, bs, D), 2, dev, dtype)
    table = torch.randperm(B * mb, generator=torch.Generator().manual_seed(1)).view(B, mb).to(torch.int32).to(dev)
    ln, count = lengths((B,), mb * bs, 7, dev), counts(B, T, 8, dev)
    nb = ((ln + bs - 1) // bs).to(torch.int32)
    q = randn((B, T, H * G, D), 3, dev, dtype)
    kd, vd = randn((B, T, H, D), 4, dev, dtype), randn((B, T, H, D), 5, dev, dtype)
    mask = tree_masks(B, T, 6).to(dev)
    out, lse = torch.full_like(q, SENTINEL), torch.full(q.shape[:3], SENTINEL, device=dev)
    kvc.kvc_decode_attn_tree_paged(q, kvc.block_pool_view(kp, vp),
                                   kvc.page_table_view(table, nb, ln, torch.zeros((B, mb), device=dev)),
                                   kvc.make_draft(kd, vd, mask=mask, count=count), scale=0.125, out=out, lse=lse)
    assert kvc.kvc_device_status() == 0
    k, v = (x[:, table.long()].permute(1, 0, 2, 3, 4).flatten(2, 3) for x in (kp, vp))
    check(out, lse, q, k, v, kd, vd, mask, ln[:, None].expand(B, H), count, 0.125, "paged")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,Hq,R,E,T,cap", [(3000, 4, 128, 32, 2, 50), (700, 16, 256, 64, 1, 200)])
def test_thousands_of_latent_sequences(dtype, B, Hq, R, E, T, cap):
    dev = cuda_or_skip()
    kvc = lib()
    q, c, cd = (randn(s, i, dev, dtype) for i, s in enumerate([(B, T, Hq, R + E), (B, cap, R + E), (B, T, R + E)]))
    mask, lens, count = tree_masks(B, T, 6).to(dev), lengths((B,), cap, 7, dev), counts(B, T, 8, dev)
    out = torch.full((B, T, Hq, R), SENTINEL, dtype=dtype, device=dev)
    lse = torch.full((B, T, Hq), SENTINEL, device=dev)
    kvc.kvc_decode_attn_latent(q, kvc.latent_cache_view(c, R), kvc.make_draft(cd, mask=mask, count=count),
                               scale=0.07, len=lens, out=out, lse=lse)
    assert kvc.kvc_device_status() == 0
    check(out, lse, q, c[:, None], c[:, None, :, :R], cd[:, :, None], cd[:, :, None, :R], mask, lens[:, None],
          count, 0.07, "latent")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_most_rows_a_pair_can_have(dtype, D):
    """64 drafted tokens of 64 query heads a KV head: 4096 rows in 32 or more row tiles."""
    dev = cuda_or_skip()
    kvc = lib()
    B, H, G, T, cap = 2, 1, 64, 64, 300
    q = randn((B, T, H * G, D), 1, dev, dtype)
    k, v = randn((B, H, cap, D), 2, dev, dtype), randn((B, H, cap, D), 3, dev, dtype)
    kd, vd = randn((B, T, H, D), 4, dev, dtype), randn((B, T, H, D), 5, dev, dtype)
    lens = torch.tensor([[cap], [129]], dtype=torch.int32, device=dev)
    mask, count = tree_masks(B, T, 6).to(dev), torch.tensor([T, 37], dtype=torch.int32, device=dev)
    out, lse = torch.full_like(q, SENTINEL), torch.full(q.shape[:3], SENTINEL, device=dev)
    kvc.kvc_decode_attn_tree(q, kvc.cache_view(k, v), kvc.make_draft(kd, vd, mask=mask, count=count),
                             scale=D ** -0.5, len=lens, out=out, lse=lse)
    assert kvc.kvc_device_status() == 0
    check(out, lse, q, k, v, kd, vd, mask, lens, count, D ** -0.5, "rows")


@pytest.mark.parametrize("dtype", TYPES)
def test_the_most_rows_a_latent_sequence_can_have(dtype):
    """64 drafted tokens of 256 heads: 16384 rows, more row tiles than the GPU has SMs."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hq, R, E, T, cap = 2, 256, 128, 64, 64, 200
    q, c, cd = (randn(s, i, dev, dtype) for i, s in enumerate([(B, T, Hq, R + E), (B, cap, R + E), (B, T, R + E)]))
    lens = torch.tensor([cap, 65], dtype=torch.int32, device=dev)
    mask, count = tree_masks(B, T, 6).to(dev), torch.tensor([41, T], dtype=torch.int32, device=dev)
    out = torch.full((B, T, Hq, R), SENTINEL, dtype=dtype, device=dev)
    lse = torch.full((B, T, Hq), SENTINEL, device=dev)
    kvc.kvc_decode_attn_latent(q, kvc.latent_cache_view(c, R), kvc.make_draft(cd, mask=mask, count=count),
                               scale=0.07, len=lens, out=out, lse=lse)
    assert kvc.kvc_device_status() == 0
    check(out, lse, q, c[:, None], c[:, None, :, :R], cd[:, :, None], cd[:, :, None, :R], mask, lens[:, None],
          count, 0.07, "rows")


@pytest.mark.parametrize("dtype", TYPES)
def test_sequences_that_share_one_cache(dtype):
    """A prompt's rows once for the whole batch (stride_b 0), for heads too (stride_h 0)."""
    dev = cuda_or_skip()
    kvc = lib()
    B, H, G, D, T, cap = 5, 2, 3, 128, 6, 700
    q = randn((B, T, H * G, D), 1, dev, dtype)
    kd, vd = randn((B, T, H, D), 4, dev, dtype), randn((B, T, H, D), 5, dev, dtype)
    mask, lens = tree_masks(B, T, 6).to(dev), lengths((B, H), cap, 7, dev)
    every = torch.full((B,), T, dtype=torch.int32, device=dev)
    for heads in (H, 1):
        k, v = (randn((1, heads, cap, D), s, dev, dtype).expand(B, H, cap, D) for s in (2, 3))
        out, lse = torch.full_like(q, SENTINEL), torch.full(q.shape[:3], SENTINEL, device=dev)
        kvc.kvc_decode_attn_tree(q, kvc.cache_view(k, v), kvc.make_draft(kd, vd, mask=mask), scale=0.1,
                                 len=lens, out=out, lse=lse)
        check(out, lse, q, k, v, kd, vd, mask, lens, every, 0.1, f"shared by {heads} heads")
    R, E, Hq = 256, 64, 8
    ql, cd = randn((B, T, Hq, R + E), 8, dev, dtype), randn((B, T, R + E), 9, dev, dtype)
    c = randn((1, cap, R + E), 10, dev, dtype).expand(B, cap, R + E)
    out = torch.full((B, T, Hq, R), SENTINEL, dtype=dtype, device=dev)
    lse = torch.full((B, T, Hq), SENTINEL, device=dev)
    kvc.kvc_decode_attn_latent(ql, kvc.latent_cache_view(c, R), kvc.make_draft(cd, mask=mask), scale=0.07,
                               len=lens[:, 0].contiguous(), out=out, lse=lse)
    check(out, lse, ql, c[:, None], c[:, None, :, :R], cd[:, :, None], cd[:, :, None, :R], mask, lens[:, :1], every,
          0.07, "latent")
    wk, wv = randn((H, D - E, R), 11, dev, dtype), randn((H, D, R), 12, dev, dtype)
    ks, vs = (torch.full((B, H, cap, D), SENTINEL, dtype=dtype, device=dev) for _ in range(2))
    kvc.kvc_latent_expand(kvc.latent_cache_view(c, R), wk, wv, kvc.cache_view(ks, vs), n_valid=cap)
    k1, v1 = (torch.full((1, H, cap, D), SENTINEL, dtype=dtype, device=dev) for _ in range(2))
    kvc.kvc_latent_expand(kvc.latent_cache_view(c[:1], R), wk, wv, kvc.cache_view(k1, v1), n_valid=cap)
    assert kvc.kvc_device_status() == 0
    assert all(torch.equal(ks[b], k1[0]) and torch.equal(vs[b], v1[0]) for b in range(B))
