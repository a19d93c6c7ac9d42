"""GPU: latent caches -- absorbed attention of one token or a draft tree, accepted rows, expansion to
per-head keys and values -- against the 64-bit definitions, and both forms against each other."""
import math

import pytest
import torch

from gpu_helpers import cuda_or_skip, lib
from tree_ref import SENTINEL, attend, chain_masks, check, compare, randn, tolerance, tree_masks

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def run_latent(kvc, q, c, R, cd, lens, mask, count=None, scale=0.08, n_valid=None):
    out = torch.full(q.shape[:3] + (R,), SENTINEL, device=q.device, dtype=q.dtype)
    lse = torch.full(q.shape[:3], SENTINEL, device=q.device)
    draft = kvc.make_draft(cd, mask=mask, count=count, n_draft=None if cd is not None else q.shape[1])
    kvc.kvc_decode_attn_latent(q, kvc.latent_cache_view(c, R), draft, scale=scale, len=lens, n_valid=n_valid,
                               out=out, lse=lse)
    return out, lse


def verify(q, c, R, cd, lens, mask, out, lse, count=None, scale=0.08, what=""):
    B, T, H, W = q.shape
    words = chain_masks(B, T) if mask is None else mask.cpu()
    for b in range(B):
        n, m = int(lens[b]), T if count is None else int(count[b])
        assert bool((out[b, m:] == SENTINEL).all()) and bool((lse[b, m:] == SENTINEL).all())
        if m == 0:
            continue
        o, z, pv, mag = attend(q[b, :m], c[b, :n], c[b, :n, :R], None if cd is None else cd[b, :m],
                               None if cd is None else cd[b, :m, :R], words[b], scale)
        check(out[b, :m], lse[b, :m], q.dtype, [(slice(None), o, z, pv, mag, W, n + m)],
              f"{what} sequence {b}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,H,R,E,T,lens", [
    (1, 1, 128, 0, 1, [0]), (1, 16, 512, 64, 1, [1000]), (2, 16, 512, 64, 1, [1, 64]),
    (3, 8, 256, 32, 5, [0, 63, 65]), (2, 128, 512, 64, 2, [300, 129]), (2, 24, 128, 8, 64, [77, 0]),
    (1, 100, 256, 64, 3, [513]), (4, 16, 512, 32, 4, [5, 0, 128, 700]), (1, 256, 128, 64, 7, [200]),
    (1, 5, 512, 0, 13, [1]), (1, 64, 256, 56, 1, [12000]), (1, 3, 512, 64, 2, [20000])])
def test_latent_matches_definition(dtype, B, H, R, E, T, lens):
    """Head counts below, at and across the row tiles, rope parts of every kind, lengths from none to
    many tiles (and one sequence split over every block)."""
    dev = cuda_or_skip()
    kvc = lib()
    seed = 7000 + H + R + T
    q = randn((B, T, H, R + E), seed, dev, dtype)
    c = randn((B, max(1, max(lens)) + 2, R + E), seed + 1, dev, dtype)
    cd = randn((B, T, R + E), seed + 2, dev, dtype)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    mask = tree_masks(B, T, seed).to(dev)
    out, lse = run_latent(kvc, q, c, R, cd, ln, mask)
    assert kvc.kvc_device_status() == 0
    verify(q, c, R, cd, ln, mask, out, lse)
    again, lse2 = run_latent(kvc, q, c, R, cd, ln, mask)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_latent_counts_garbage_strides_and_chain(dtype):
    """Padded rows and a strided batch, counts from none to all, garbage wherever nothing may be read,
    no mask, cache only, n_valid."""
    dev = cuda_or_skip()
    kvc = lib()
    B, H, R, E, T, cap = 4, 20, 256, 32, 6, 200
    buf = torch.full((B, cap + 5, R + E + 16), NAN, device=dev, dtype=dtype)
    c = buf[:, 2:cap + 2, :R + E]
    c.copy_(randn((B, cap, R + E), 1, dev, dtype))
    q = randn((B, T, H, R + E), 2, dev, dtype)
    cd = randn((B, T, R + E), 3, dev, dtype)
    ln = torch.tensor([0, 130, 199, 64], dtype=torch.int32, device=dev)
    count = torch.tensor([6, 0, 3, 1], dtype=torch.int32, device=dev)
    for b in range(B):
        c[b, int(ln[b]):] = INF
        cd[b, int(count[b]):] = NAN
    mask = tree_masks(B, T, 3)
    mask[0] &= ~(1 << 4)
    mask[0, 1] = 0
    cd[0, 4] = NAN
    cd[2, 1, 7] = -INF                   # as a value and as a key of the rows that see it
    mask[2, 2] = 1 << 2
    mask[2, 0] = 1
    mask = mask.to(dev)
    out, lse = run_latent(kvc, q, c, R, cd, ln, mask, count=count)
    assert kvc.kvc_device_status() == 0
    sees = [t for t in range(3) if (int(mask[2, t]) >> 1) & 1]
    keep = torch.ones(out.shape[:2], dtype=torch.bool)
    for t in sees:                       # infinite logits there: only that nothing leaks from them
        keep[2, t] = False
    clean = cd.clone()
    clean[2, 1, 7] = 0
    ok = out.clone()
    lk = lse.clone()
    ref_out, ref_lse = run_latent(kvc, q, c, R, clean, ln, mask, count=count)
    ok[2, sees], lk[2, sees] = ref_out[2, sees], ref_lse[2, sees]
    verify(q, c, R, clean, ln, mask, ok, lk, count=count)
    c.copy_(randn((B, cap, R + E), 1, dev, dtype))
    cd = randn((B, T, R + E), 3, dev, dtype)
    out, lse = run_latent(kvc, q, c, R, cd, ln, None)
    verify(q, c, R, cd, ln, None, out, lse, what="chain")
    for n in (0, 1, 200):
        full = torch.full((B,), n, dtype=torch.int32)
        out, lse = run_latent(kvc, q, c, R, None, None, None, n_valid=n)
        verify(q, c, R, None, full, None, out, lse, what=f"cache only {n}")


@pytest.mark.parametrize("B,H,R,E,T,cap,lens", [
    (4, 20, 256, 32, 6, 900, [0, 830, 899, 64]), (4, 16, 512, 64, 2, 2000, [2000, 1, 0, 1217]),
    (170, 16, 512, 64, 1, 130, [0, 1, 64, 65, 130]), (320, 20, 128, 0, 5, 100, [100, 0, 37])])
def test_latent_garbage_in_split_and_whole_sequences(B, H, R, E, T, cap, lens):
    """Counts from none to all and garbage wherever nothing may be read, in few sequences that are split
    and in more short ones than blocks."""
    dev = cuda_or_skip()
    kvc = lib()
    dtype = torch.bfloat16
    q, c = randn((B, T, H, R + E), 31, dev, dtype), randn((B, cap, R + E), 32, dev, dtype)
    cd = randn((B, T, R + E), 33, dev, dtype)
    ln = torch.tensor([lens[b % len(lens)] for b in range(B)], dtype=torch.int32, device=dev)
    count = torch.tensor([(T, 0, T, 1, T // 2)[b % 5] for b in range(B)], dtype=torch.int32, device=dev)
    for b in range(B):
        c[b, int(ln[b]):] = (INF, NAN)[b % 2]
        cd[b, int(count[b]):] = NAN
    mask = tree_masks(B, T, 34)
    mask[0, 0] = 0
    out, lse = run_latent(kvc, q, c, R, cd, ln, mask.to(dev), count=count)
    assert kvc.kvc_device_status() == 0
    verify(q, c, R, cd, ln, mask, out, lse, count=count)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,H,R,E,D,cap,lens", [
    (1, 1, 128, 0, 64, 5, [5]), (2, 3, 256, 32, 64, 130, [0, 129]), (2, 8, 512, 64, 128, 300, [300, 1]),
    (1, 5, 512, 32, 256, 257, [257]), (3, 2, 128, 56, 128, 64, [64, 63, 0]), (1, 32, 256, 64, 128, 600, [511]),
    (1, 2, 512, 64, 256, 129, [128])])
def test_expand_matches_definition(dtype, B, H, R, E, D, cap, lens):
    """Rows of every head to the length, later slots as they were, strided destination."""
    dev = cuda_or_skip()
    kvc = lib()
    c = randn((B, cap, R + E), 1, dev, dtype)
    for b in range(B):
        c[b, lens[b]:] = NAN
    wk, wv = (randn((H, D - E, R), 2, dev, dtype) / math.sqrt(R)), (randn((H, D, R), 3, dev, dtype) / math.sqrt(R))
    wk, wv = wk.to(dtype), wv.to(dtype)
    buf = torch.full((B, cap + 3, H, 2, D), SENTINEL, device=dev, dtype=dtype)
    k, v = buf[:, :, :, 0].transpose(1, 2), buf[:, :, :, 1].transpose(1, 2)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    kvc.kvc_latent_expand(kvc.latent_cache_view(c, R), wk, wv, kvc.cache_view(k, v), len=ln)
    assert kvc.kvc_device_status() == 0
    eps = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    for b in range(B):
        n = lens[b]
        assert bool((k[b, :, n:] == SENTINEL).all()) and bool((v[b, :, n:] == SENTINEL).all())
        lat = c[b, :n, :R].double()
        assert torch.equal(k[b, :, :n, D - E:], c[b, :n, R:].expand(H, n, E))
        for got, w in ((k[b, :, :n, :D - E], wk), (v[b, :, :n], wv)):
            ref = torch.einsum("sr,hir->hsi", lat, w.double())
            # R products accumulated in fp32 (R * 2^-23 of their magnitudes), one rounding
            mag = torch.einsum("sr,hir->hsi", lat.abs(), w.double().abs())
            compare(got, ref, eps * ref.abs() + (1 + eps) * R * 2.0 ** -23 * mag + 1e-30, f"expand {b}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_accept_latent(dtype):
    dev = cuda_or_skip()
    kvc = lib()
    B, R, E, T, cap = 3, 128, 24, 9, 40
    c, cd = randn((B, cap, R + E), 1, dev, dtype), randn((B, T, R + E), 2, dev, dtype)
    ln = torch.tensor([0, 35, 31], dtype=torch.int32, device=dev)
    path = torch.stack([torch.randperm(T, generator=torch.Generator().manual_seed(i)) for i in range(B)])
    path = path.to(torch.int32).to(dev)
    n = torch.tensor([4, 6, 9], dtype=torch.int32, device=dev)
    want = c.clone()
    for b in (0, 2):
        a, m = int(ln[b]), int(n[b])
        want[b, a:a + m] = cd[b, path[b, :m].long()]
    kvc.kvc_latent_accept(kvc.latent_cache_view(c, R), ln, kvc.make_draft(cd), path, n)
    assert kvc.kvc_device_status() == 1                     # KVC_DEV_TAIL_FULL: 35 + 6 > 40
    assert torch.equal(c, want) and ln.tolist() == [4, 35, 40]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_absorbed_and_expanded_forms_agree(dtype):
    """The run a program makes: drafts, latent attention, acceptance, three times; at each step the
    expanded cache gives the same attention through kvc_decode_attn_tree."""
    dev = cuda_or_skip()
    kvc = lib()
    B, H, R, E, D, T, cap = 2, 8, 256, 64, 128, 6, 120
    wk = (randn((H, D - E, R), 2, dev, torch.float32) / math.sqrt(R)).to(dtype)
    wv = (randn((H, D, R), 3, dev, torch.float32) / math.sqrt(R)).to(dtype)
    c = torch.full((B, cap, R + E), NAN, device=dev, dtype=dtype)
    ln = torch.tensor([70, 9], dtype=torch.int32, device=dev)
    for b in range(B):
        c[b, :int(ln[b])] = randn((int(ln[b]), R + E), 60 + b, dev, dtype)
    scale = 1 / math.sqrt(D)
    for step in range(3):
        q = randn((B, T, H, D), 10 + step, dev, dtype)
        cd = randn((B, T, R + E), 20 + step, dev, dtype)
        mask = tree_masks(B, T, step).to(dev)
        qa = torch.cat([torch.einsum("bthi,hir->bthr", q[..., :D - E].float(), wk.float()),
                        q[..., D - E:].float()], dim=3).to(dtype)
        out, lse = run_latent(kvc, qa, c, R, cd, ln, mask, scale=scale)
        verify(qa, c, R, cd, ln, mask, out, lse, scale=scale)
        # expanded: the cache and the drafts through the same matrices
        k, v = (torch.zeros((B, H, cap, D), device=dev, dtype=dtype) for _ in range(2))
        kvc.kvc_latent_expand(kvc.latent_cache_view(c, R), wk, wv, kvc.cache_view(k, v), len=ln)
        kd, vd = (torch.zeros((B, H, T, D), device=dev, dtype=dtype) for _ in range(2))
        kvc.kvc_latent_expand(kvc.latent_cache_view(cd, R), wk, wv, kvc.cache_view(kd, vd), n_valid=T)
        draft = kvc.make_draft(kd.transpose(1, 2).contiguous(), vd.transpose(1, 2).contiguous(), mask=mask)
        exp = kvc.kvc_decode_attn_tree(q, kvc.cache_view(k, v), draft, scale=scale,
                                       len=ln[:, None].expand(B, H).contiguous())
        head = torch.einsum("bthr,hir->bthi", out.double(), wv.double())
        # Either form is off the exact attention by its operator's own bound; besides, the absorbed
        # queries are rounded (their logits by eps * scale * sum |q' c|), and so are the expanded
        # keys (eps * scale * sum |q k|) and values (eps * sum p |v|).  A logit off by d moves
        # the output by at most 2 d sum p |v|.
        eps = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -22
        for b in range(B):
            m = int(ln[b])
            o, z, pv, mag = attend(qa[b], c[b, :m], c[b, :m, :R], cd[b], cd[b, :, :R], mask[b].cpu(), scale)
            t_lat = tolerance(dtype, R + E, m + T, pv, mag, o, z)[0] + 2 * eps * mag[..., None] * pv
            t_head = torch.einsum("thr,hir->thi", t_lat, wv.double().abs())
            for h in range(H):
                o, z, pv, mag = attend(q[b, :, h:h + 1], k[b, h, :m], v[b, h, :m], kd[b, h], vd[b, h],
                                       mask[b].cpu(), scale)
                t_exp = tolerance(dtype, D, m + T, pv, mag, o, z)[0] + (2 * eps * mag[..., None] + eps) * pv
                compare(exp[b, :, h], head[b, :, h], t_exp[:, 0] + t_head[:, h], f"forms {step} {b} {h}")
        n = torch.tensor([3, 2], dtype=torch.int32, device=dev)
        path = torch.arange(T, dtype=torch.int32, device=dev).repeat(B, 1)
        kvc.kvc_latent_accept(kvc.latent_cache_view(c, R), ln, kvc.make_draft(cd), path, n)
    assert ln.tolist() == [79, 15] and kvc.kvc_device_status() == 0


def test_latent_in_a_graph():
    dev = cuda_or_skip()
    kvc = lib()
    B, H, R, E, T, cap = 2, 16, 512, 64, 2, 900
    q, c = randn((B, T, H, R + E), 1, dev, torch.bfloat16), randn((B, cap, R + E), 2, dev, torch.bfloat16)
    cd = randn((B, T, R + E), 3, dev, torch.bfloat16)
    ln = torch.tensor([5, 5], dtype=torch.int32, device=dev)
    cache, draft = kvc.latent_cache_view(c, R), kvc.make_draft(cd)
    ws = kvc.latent_workspace(B, H, R, E, T, q.dtype, dev)
    out, lse = torch.empty((B, T, H, R), device=dev, dtype=q.dtype), torch.empty((B, T, H), device=dev)
    path = torch.arange(T, dtype=torch.int32, device=dev).repeat(B, 1)
    n = torch.full((B,), T, dtype=torch.int32, device=dev)
    kvc.kvc_decode_attn_latent(q, cache, draft, scale=0.05, len=ln, out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvc.kvc_decode_attn_latent(q, cache, draft, scale=0.05, len=ln, out=out, lse=lse, ws=ws)
        kvc.kvc_latent_accept(cache, ln, draft, path, n)
    for step in range(4):
        if step == 2:
            ln.copy_(torch.tensor([700, 64], dtype=torch.int32))
        cd.copy_(randn((B, T, R + E), 30 + step, dev, torch.bfloat16))
        before = ln.clone()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ln, before + T)
        verify(q, c, R, cd, before, None, out, lse, scale=0.05, what=f"replay {step}")
        for b in range(B):
            assert torch.equal(c[b, int(before[b]):int(ln[b])], cd[b])
