"""GPU: attention of a tree of drafted tokens over contiguous and paged caches, accepted paths,
against the 64-bit definitions, and a verification loop of both together."""
import math

import pytest
import torch

from gpu_helpers import cuda_or_skip, lib
from tree_ref import SENTINEL, attend, chain_masks, check, compare, randn, tolerance, tree_masks

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def run_tree(kvc, q, k, v, kd, vd, lens, mask, count=None, scale=None, n_valid=None, ws=None):
    """Call over sentinel-filled outputs; returns out, lse."""
    out = torch.full_like(q, SENTINEL)
    lse = torch.full(q.shape[:3], SENTINEL, device=q.device)
    draft = kvc.make_draft(kd, vd, mask=mask, count=count, n_draft=None if kd is not None else q.shape[1])
    scale = 1 / math.sqrt(q.shape[3]) if scale is None else scale
    kvc.kvc_decode_attn_tree(q, kvc.cache_view(k, v), draft, scale=scale, len=lens, n_valid=n_valid,
                             out=out, lse=lse, ws=ws)
    return out, lse


def verify(q, k, v, kd, vd, lens, mask, out, lse, count=None, scale=None, what=""):
    B, T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    words = (chain_masks(B, T) if mask is None else mask.cpu())
    for b in range(B):
        c = T if count is None else int(count[b])
        assert bool((out[b, c:] == SENTINEL).all()) and bool((lse[b, c:] == SENTINEL).all()), \
            f"{what}: rows behind the count were written"
        for h in range(Hkv if c else 0):
            n = int(lens[b, h]) if lens.dim() == 2 else int(lens[b])
            o, z, pv, mag = attend(q[b, :c, h * G:(h + 1) * G], k[b, h, :n], v[b, h, :n],
                                   None if kd is None else kd[b, :c, h],
                                   None if kd is None else vd[b, :c, h], words[b], scale)
            check(out[b, :c, h * G:(h + 1) * G], lse[b, :c, h * G:(h + 1) * G], q.dtype,
                  [(slice(None), o, z, pv, mag, D, n + c)], f"{what} sequence {b} head {h}")


CASES = [
    # B, Hkv, G, D, T, lens of the rows (cycled)
    (1, 1, 1, 64, 1, [0]),
    (2, 1, 1, 64, 1, [1, 65]),
    (1, 2, 4, 64, 4, [128, 127]),
    (3, 2, 3, 64, 21, [0, 1, 129, 300, 64, 63]),
    (2, 2, 8, 64, 64, [200, 1000]),
    (1, 1, 1, 128, 1, [2500]),
    (2, 2, 4, 128, 16, [0, 5, 128, 641]),
    (2, 3, 8, 128, 9, [127, 129, 1, 0, 400, 256]),
    (2, 1, 6, 128, 64, [511, 77]),
    (1, 2, 64, 128, 3, [90, 700]),
    (5, 1, 2, 128, 33, [3, 128, 1024, 0, 257]),
    (2, 2, 6, 256, 11, [0, 64, 65, 513]),
    (1, 1, 4, 256, 37, [1300]),
    (2, 2, 1, 256, 2, [63, 1, 64, 129]),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_tree_matches_definition(dtype, case):
    """Random trees over ragged lengths (none, one, around the tiles' edges), any group size."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv, G, D, T, ls = CASES[case]
    seed = 4000 + case
    lens = torch.tensor([ls[i % len(ls)] for i in range(B * Hkv)], dtype=torch.int32,
                        device=dev).view(B, Hkv)
    cap = max(1, max(ls)) + 3
    q = randn((B, T, Hkv * G, D), seed, dev, dtype)
    k, v = randn((B, Hkv, cap, D), seed + 1, dev, dtype), randn((B, Hkv, cap, D), seed + 2, dev, dtype)
    kd, vd = randn((B, T, Hkv, D), seed + 3, dev, dtype), randn((B, T, Hkv, D), seed + 4, dev, dtype)
    mask = tree_masks(B, T, seed).to(dev)
    out, lse = run_tree(kvc, q, k, v, kd, vd, lens, mask)
    assert kvc.kvc_device_status() == 0
    verify(q, k, v, kd, vd, lens, mask, out, lse)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tree_ragged_counts_masks_and_garbage(dtype, D):
    """Counts from none to all, rows that see nothing, and NaN / infinities wherever nothing may be
    read: slots behind the length, drafts behind the count, drafts a row does not see."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv, G, T, cap = 4, 2, 2, 13, 300
    q = randn((B, T, Hkv * G, D), 1, dev, dtype)
    k, v = randn((B, Hkv, cap, D), 2, dev, dtype), randn((B, Hkv, cap, D), 3, dev, dtype)
    kd, vd = randn((B, T, Hkv, D), 4, dev, dtype), randn((B, T, Hkv, D), 5, dev, dtype)
    lens = torch.tensor([[0, 0], [130, 7], [256, 299], [5, 128]], dtype=torch.int32, device=dev)
    count = torch.tensor([13, 0, 6, 1], dtype=torch.int32, device=dev)
    for b in range(B):
        for h in range(Hkv):
            n = int(lens[b, h])
            k[b, h, n:], v[b, h, n:] = NAN, INF
        kd[b, int(count[b]):], vd[b, int(count[b]):] = INF, NAN
    mask = tree_masks(B, T, 9)
    mask[0, 2] = 0                       # sees nothing at all: sequence 0 has no slots either
    mask[2, 3] = 0                       # sees the cache only
    kd[0, 7], vd[0, 7] = NAN, NAN        # a drafted token that no row sees (but counts)
    mask[0] &= ~(1 << 7)
    vd[2, 4, 1, 3] = INF                 # seen by some rows: infinity there, not elsewhere
    vd[2, 4, 1, 5] = NAN
    mask[2, 5] = 1 << 5
    mask = mask.to(dev)
    out, lse = run_tree(kvc, q, k, v, kd, vd, lens, mask, count=count)
    assert kvc.kvc_device_status() == 0
    verify(q, k, v, kd, vd, lens, mask, out, lse, count=count)
    assert bool((out[0, 2] == 0).all()) and bool((lse[0, 2] == -INF).all())


@pytest.mark.parametrize("D,T", [(64, 13), (64, 64), (128, 13), (128, 64), (256, 13), (256, 64)])
def test_tree_garbage_in_split_pairs(D, T):
    """The same in a cache whose capacity lets pairs be split, with one and with two row tiles of the
    tensor cores: parts without drafts, with nothing but drafts, non-finite drafted values in both."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv, G, cap, dtype = 4, 2, 3, 1700, torch.bfloat16
    q = randn((B, T, Hkv * G, D), 11, dev, dtype)
    k, v = randn((B, Hkv, cap, D), 12, dev, dtype), randn((B, Hkv, cap, D), 13, dev, dtype)
    kd, vd = randn((B, T, Hkv, D), 14, dev, dtype), randn((B, T, Hkv, D), 15, dev, dtype)
    lens = torch.tensor([[0, 1699], [130, 7], [1280, 1281], [5, 128]], dtype=torch.int32, device=dev)
    count = torch.tensor([T, 0, 6, 1], dtype=torch.int32, device=dev)
    for b in range(B):
        for h in range(Hkv):
            n = int(lens[b, h])
            k[b, h, n:], v[b, h, n:] = INF, NAN
        kd[b, int(count[b]):], vd[b, int(count[b]):] = NAN, INF
    mask = tree_masks(B, T, 19)
    mask[0, 2] = 0
    mask[2, 3] = 0
    vd[0, 5, 1, 9] = -INF                # in a pair of many parts
    vd[0, 6, 1, D - 1] = NAN
    vd[2, 4, 1, 3] = INF
    mask[2, 5] = 1 << 5
    mask = mask.to(dev)
    out, lse = run_tree(kvc, q, k, v, kd, vd, lens, mask, count=count)
    assert kvc.kvc_device_status() == 0
    verify(q, k, v, kd, vd, lens, mask, out, lse, count=count)


@pytest.mark.parametrize("D,G,T", [(64, 2, 3), (128, 4, 40), (128, 1, 5), (256, 2, 3), (256, 5, 33)])
@pytest.mark.parametrize("drafts", [True, False])
def test_tree_many_short_pairs(D, G, T, drafts):
    """More short pairs than blocks, which whole blocks take pair by pair: ragged lengths with empty
    pairs at either end, sequences without drafted tokens, more than one row tile."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv, cap, dtype = 59, 8, 150, torch.bfloat16
    q = randn((B, T, Hkv * G, D), 21, dev, dtype)
    k, v = randn((B, Hkv, cap, D), 22, dev, dtype), randn((B, Hkv, cap, D), 23, dev, dtype)
    kd, vd = randn((B, T, Hkv, D), 24, dev, dtype), randn((B, T, Hkv, D), 25, dev, dtype)
    gen = torch.Generator().manual_seed(26)
    lens = torch.randint(0, cap + 1, (B, Hkv), generator=gen, dtype=torch.int32)
    lens[0], lens[-1], lens[20] = 0, 0, cap
    count = torch.randint(0, T + 1, (B,), generator=gen, dtype=torch.int32)
    count[0], count[1], count[-1] = 0, T, 0
    lens, count = lens.to(dev), count.to(dev)
    mask = tree_masks(B, T, 27).to(dev)
    if not drafts:
        kd = vd = mask = None
    out, lse = run_tree(kvc, q, k, v, kd, vd, lens, mask, count=count)
    assert kvc.kvc_device_status() == 0
    verify(q, k, v, kd, vd, lens, mask, out, lse, count=count)
    lens[3, 5], count[7] = cap + 9, -2   # recorded, and clamped
    out, lse = run_tree(kvc, q, k, v, kd, vd, lens, mask, count=count)
    assert kvc.kvc_device_status() == 5                     # KVC_DEV_BAD_LENGTH
    lens[3, 5], count[7] = cap, 0
    verify(q, k, v, kd, vd, lens, mask, out, lse, count=count)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tree_chain_cache_only_and_n_valid(dtype):
    """No mask: a chain.  No drafted rows: the cache only.  n_valid instead of lengths, also 0."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv, G, D, T, cap = 2, 2, 4, 128, 7, 333
    q = randn((B, T, Hkv * G, D), 1, dev, dtype)
    k, v = randn((B, Hkv, cap, D), 2, dev, dtype), randn((B, Hkv, cap, D), 3, dev, dtype)
    kd, vd = randn((B, T, Hkv, D), 4, dev, dtype), randn((B, T, Hkv, D), 5, dev, dtype)
    for n in (0, 1, 300, 333):
        full = torch.full((B, Hkv), n, dtype=torch.int32, device=dev)
        out, lse = run_tree(kvc, q, k, v, kd, vd, None, None, n_valid=n)
        verify(q, k, v, kd, vd, full, None, out, lse, what=f"chain {n}")
        out, lse = run_tree(kvc, q, k, v, None, None, full, None)
        verify(q, k, v, None, None, full, None, out, lse, what=f"cache only {n}")
    assert kvc.kvc_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_tree_scales(dtype, scale):
    """A zero scale (uniform weights), a negative one, and one whose logits span hundreds."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv, G, D, T, cap = 1, 2, 4, 64, 5, 400
    q = randn((B, T, Hkv * G, D), 11, dev, dtype)
    k, v = randn((B, Hkv, cap, D), 12, dev, dtype), randn((B, Hkv, cap, D), 13, dev, dtype)
    kd, vd = randn((B, T, Hkv, D), 14, dev, dtype), randn((B, T, Hkv, D), 15, dev, dtype)
    k[:, :, 390:] *= 4                   # the maximum comes late: the running state is rescaled
    lens = torch.full((B, Hkv), cap, dtype=torch.int32, device=dev)
    mask = tree_masks(B, T, 3).to(dev)
    out, lse = run_tree(kvc, q, k, v, kd, vd, lens, mask, scale=scale)
    verify(q, k, v, kd, vd, lens, mask, out, lse, scale=scale)


def test_tree_rising_maximum():
    """Keys that grow along the cache: the running maximum rises in every tile, by little and by
    much, so partial sums are rescaled throughout."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv, G, D, T, cap = 1, 1, 4, 128, 40, 3000
    q = randn((B, T, Hkv * G, D), 21, dev, torch.bfloat16)
    k, v = randn((B, Hkv, cap, D), 22, dev, torch.bfloat16), randn((B, Hkv, cap, D), 23, dev, torch.bfloat16)
    k *= torch.linspace(0.1, 12, cap, device=dev)[None, None, :, None].to(k.dtype)
    kd, vd = randn((B, T, Hkv, D), 24, dev, torch.bfloat16), randn((B, T, Hkv, D), 25, dev, torch.bfloat16)
    lens = torch.full((B, Hkv), cap, dtype=torch.int32, device=dev)
    mask = tree_masks(B, T, 4).to(dev)
    out, lse = run_tree(kvc, q, k, v, kd, vd, lens, mask)
    verify(q, k, v, kd, vd, lens, mask, out, lse)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tree_one_long_row_is_split(dtype):
    """One head, one token, a long cache: every block takes a piece, the merge joins them; twice the
    same bits."""
    dev = cuda_or_skip()
    kvc = lib()
    for D, T, n in ((128, 1, 40001), (64, 3, 30000), (256, 2, 20011)):
        q = randn((1, T, 1, D), 1, dev, dtype)
        k, v = randn((1, 1, n, D), 2, dev, dtype), randn((1, 1, n, D), 3, dev, dtype)
        kd, vd = randn((1, T, 1, D), 4, dev, dtype), randn((1, T, 1, D), 5, dev, dtype)
        lens = torch.tensor([[n]], dtype=torch.int32, device=dev)
        mask = tree_masks(1, T, 5).to(dev)
        out, lse = run_tree(kvc, q, k, v, kd, vd, lens, mask)
        verify(q, k, v, kd, vd, lens, mask, out, lse)
        again, lse2 = run_tree(kvc, q, k, v, kd, vd, lens, mask)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tree_strided_cache(dtype):
    """Slots wider than a head, heads inside slots, and a view into a larger buffer."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv, G, D, T, cap = 2, 3, 2, 128, 6, 270
    buf = randn((B, cap, Hkv, 2, D), 31, dev, dtype)       # [b][slot][head][k or v][d]
    k, v = buf[:, :, :, 0].transpose(1, 2), buf[:, :, :, 1].transpose(1, 2)
    q = randn((B, T, Hkv * G, D), 32, dev, dtype)
    kd, vd = randn((B, T, Hkv, D), 34, dev, dtype), randn((B, T, Hkv, D), 35, dev, dtype)
    lens = torch.tensor([[270, 129, 1], [0, 200, 128]], dtype=torch.int32, device=dev)
    mask = tree_masks(B, T, 6).to(dev)
    out, lse = run_tree(kvc, q, k, v, kd, vd, lens, mask)
    verify(q, k, v, kd, vd, lens, mask, out, lse)


def test_tree_offsets_past_32_bits():
    """Heads more than 2^32 bytes (and 2^31 elements) apart."""
    dev = cuda_or_skip()
    kvc = lib()
    D, cap, far = 64, 200, 2 ** 31 + 8 * 64
    q = randn((1, 3, 4, D), 1, dev, torch.bfloat16)
    kd, vd = randn((1, 3, 2, D), 4, dev, torch.bfloat16), randn((1, 3, 2, D), 5, dev, torch.bfloat16)
    buf = torch.empty(far + 2 * cap * D, dtype=torch.bfloat16, device=dev)
    k = buf.as_strided((1, 2, cap, D), (far * 2, far, D, 1))
    v = buf[cap * D:].as_strided((1, 2, cap, D), (far * 2, far, D, 1))
    k.copy_(randn((1, 2, cap, D), 2, dev, torch.bfloat16))
    v.copy_(randn((1, 2, cap, D), 3, dev, torch.bfloat16))
    lens = torch.tensor([[cap, cap]], dtype=torch.int32, device=dev)
    mask = tree_masks(1, 3, 5).to(dev)
    out, lse = run_tree(kvc, q, k, v, kd, vd, lens, mask)
    verify(q, k, v, kd, vd, lens, mask, out, lse)
    path = torch.tensor([[0, 2, 1]], dtype=torch.int32, device=dev)
    n = torch.tensor([2], dtype=torch.int32, device=dev)
    lens.fill_(10)
    kvc.kvc_tree_accept(kvc.cache_view(k, v), lens, kvc.make_draft(kd, vd), path, n)
    assert torch.equal(k[0, 1, 10:12], kd[0, [0, 2], 1]) and torch.equal(v[0, 1, 10:12], vd[0, [0, 2], 1])
    assert lens.tolist() == [[12, 12]]


def paged_setup(dev, dtype, B, Hkv, D, bs, lens, seed, spare=5):
    mb = max(1, max(-(-n // bs) for n in lens)) + 1
    n_pool = B * mb + spare
    kp, vp = randn((Hkv, n_pool, bs, D), seed, dev, dtype), randn((Hkv, n_pool, bs, D), seed + 1, dev, dtype)
    perm = torch.randperm(n_pool, generator=torch.Generator().manual_seed(seed))
    table = torch.full((B, mb), -1, dtype=torch.int32)
    used = 0
    for b, n in enumerate(lens):
        nb = -(-n // bs)
        table[b, :nb] = perm[used:used + nb].to(torch.int32)
        used += nb
    free = perm[used:].to(torch.int32).to(dev)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    nb = torch.tensor([-(-n // bs) for n in lens], dtype=torch.int32, device=dev)
    return kp, vp, table.to(dev), nb, ln, torch.zeros((B, mb), device=dev), free


def logical(pool, table, n, bs, b):
    """[Hkv, n, D] of sequence b."""
    nb = -(-n // bs)
    return pool[:, table[b, :nb].long()].flatten(1, 2)[:, :n]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,G,T,bs", [(128, 1, 8, 32), (128, 4, 5, 16), (64, 2, 17, 64), (256, 6, 3, 32),
                                      (128, 2, 40, 128), (64, 1, 1, 256), (128, 1, 3, 7), (256, 1, 2, 128),
                                      (64, 8, 30, 8), (128, 1, 2, 24), (256, 2, 5, 64)])
def test_tree_paged_matches_definition(dtype, D, G, T, bs):
    """Shuffled pages, lengths that end inside pages and tiles, unused table entries left invalid,
    any block size."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv = 5, 2
    lens = [0, 1, 3 * bs, 2 * bs + max(1, bs // 2), 400]
    kp, vp, table, nb, ln, score, _ = paged_setup(dev, dtype, B, Hkv, D, bs, lens, 50 + D + bs)
    q = randn((B, T, Hkv * G, D), 1, dev, dtype)
    kd, vd = randn((B, T, Hkv, D), 4, dev, dtype), randn((B, T, Hkv, D), 5, dev, dtype)
    mask = tree_masks(B, T, 7).to(dev)
    out, lse = torch.full_like(q, SENTINEL), torch.full(q.shape[:3], SENTINEL, device=dev)
    kvc.kvc_decode_attn_tree_paged(q, kvc.block_pool_view(kp, vp),
                                   kvc.page_table_view(table, nb, ln, score),
                                   kvc.make_draft(kd, vd, mask=mask), scale=1 / math.sqrt(D), out=out,
                                   lse=lse)
    assert kvc.kvc_device_status() == 0
    for b in range(B):
        kc, vc = logical(kp, table, lens[b], bs, b)[None], logical(vp, table, lens[b], bs, b)[None]
        verify(q[b:b + 1], kc, vc, kd[b:b + 1], vd[b:b + 1],
               torch.full((1, Hkv), lens[b], dtype=torch.int32), mask[b:b + 1], out[b:b + 1],
               lse[b:b + 1], what=f"paged {b}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tree_paged_bad_entries_are_recorded(dtype):
    """A table entry outside the pool: the code is recorded, block 0 stands in, other sequences
    are right."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv, D, bs, T, lens = 2, 1, 128, 32, 4, [100, 70]
    kp, vp, table, nb, ln, score, _ = paged_setup(dev, dtype, B, Hkv, D, bs, lens, 3)
    table[0, 1] = kp.shape[1]
    table[0, 2] = -7
    q = randn((B, T, 2, D), 1, dev, dtype)
    kd, vd = randn((B, T, Hkv, D), 4, dev, dtype), randn((B, T, Hkv, D), 5, dev, dtype)
    mask = tree_masks(B, T, 7).to(dev)
    out, lse = torch.full_like(q, SENTINEL), torch.full(q.shape[:3], SENTINEL, device=dev)
    kvc.kvc_decode_attn_tree_paged(q, kvc.block_pool_view(kp, vp),
                                   kvc.page_table_view(table, nb, ln, score),
                                   kvc.make_draft(kd, vd, mask=mask), scale=0.1, out=out, lse=lse)
    assert kvc.kvc_device_status() == 9                     # KVC_DEV_BAD_BLOCK
    table[0, 1:3] = 0
    for b in range(B):
        kc, vc = logical(kp, table, lens[b], bs, b)[None], logical(vp, table, lens[b], bs, b)[None]
        verify(q[b:b + 1], kc, vc, kd[b:b + 1], vd[b:b + 1],
               torch.full((1, Hkv), lens[b], dtype=torch.int32), mask[b:b + 1], out[b:b + 1],
               lse[b:b + 1], scale=0.1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tree_lengths_and_counts_out_of_range(dtype):
    """Lengths and counts outside their ranges are recorded and clamped."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv, D, T, cap = 2, 2, 64, 5, 140
    q = randn((B, T, Hkv, D), 1, dev, dtype)
    k, v = randn((B, Hkv, cap, D), 2, dev, dtype), randn((B, Hkv, cap, D), 3, dev, dtype)
    kd, vd = randn((B, T, Hkv, D), 4, dev, dtype), randn((B, T, Hkv, D), 5, dev, dtype)
    lens = torch.tensor([[-3, 100], [cap + 9, 2 ** 31 - 1]], dtype=torch.int32, device=dev)
    mask = tree_masks(B, T, 1).to(dev)
    out, lse = run_tree(kvc, q, k, v, kd, vd, lens, mask)
    assert kvc.kvc_device_status() == 5                     # KVC_DEV_BAD_LENGTH
    verify(q, k, v, kd, vd, lens.clamp(0, cap), mask, out, lse)
    lens.clamp_(0, cap)
    count = torch.tensor([-1, 99], dtype=torch.int32, device=dev)
    out, lse = run_tree(kvc, q, k, v, kd, vd, lens, mask, count=count)
    assert kvc.kvc_device_status() == 5
    verify(q, k, v, kd, vd, lens, mask, out, lse, count=count.clamp(0, T))


def test_tree_in_graphs_and_streams():
    """Captured once and replayed as lengths, masks and inputs change; two captured graphs share
    one workspace in turn; two streams run at once with a workspace each."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv, G, D, T, cap = 2, 2, 4, 128, 12, 2000
    Hq = Hkv * G
    q = randn((B, T, Hq, D), 1, dev, torch.bfloat16)
    k, v = randn((B, Hkv, cap, D), 2, dev, torch.bfloat16), randn((B, Hkv, cap, D), 3, dev, torch.bfloat16)
    kd, vd = randn((B, T, Hkv, D), 4, dev, torch.bfloat16), randn((B, T, Hkv, D), 5, dev, torch.bfloat16)
    lens = torch.full((B, Hkv), 100, dtype=torch.int32, device=dev)
    mask = tree_masks(B, T, 1).to(dev)
    ws = kvc.tree_workspace(B, Hq, Hkv, D, T, q.dtype, dev)
    ws.fill_(0xff)                                          # a workspace need not be cleared
    run_tree(kvc, q, k, v, kd, vd, lens, mask, ws=ws)
    torch.cuda.synchronize()
    graphs, outs = [], []
    q2 = randn((B, T, Hq, D), 77, dev, torch.bfloat16)
    for x in (q, q2):
        g = torch.cuda.CUDAGraph()
        out, lse = torch.empty_like(x), torch.empty(x.shape[:3], device=dev)
        draft, cache = kvc.make_draft(kd, vd, mask=mask), kvc.cache_view(k, v)
        with torch.cuda.graph(g):
            kvc.kvc_decode_attn_tree(x, cache, draft, scale=D ** -0.5, len=lens, out=out, lse=lse, ws=ws)
        graphs.append(g)
        outs.append((x, out, lse, draft, cache))
    for step, n in enumerate((100, 0, 1777, 2000, 3)):
        lens.copy_(torch.tensor([[n, max(0, n - 5)], [n // 2, n // 3]], dtype=torch.int32))
        mask.copy_(tree_masks(B, T, 30 + step))
        kd.copy_(randn((B, T, Hkv, D), 40 + step, dev, torch.bfloat16))
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for x, out, lse, _, _ in outs:
            verify(x, k, v, kd, vd, lens, mask, out, lse, what=f"replay {step}")
    lens.fill_(1500)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    torch.cuda.synchronize()
    for x, s in zip((q, q2), streams):
        with torch.cuda.stream(s):
            w = kvc.tree_workspace(B, Hq, Hkv, D, T, x.dtype, dev)
            got.append([run_tree(kvc, x, k, v, kd, vd, lens, mask, ws=w) for _ in range(5)] + [w])
    torch.cuda.synchronize()
    for x, rs in zip((q, q2), got):
        for out, lse in rs[:-1]:
            verify(x, k, v, kd, vd, lens, mask, out, lse)
    assert kvc.kvc_device_status() == 0


# --------------------------------------------------------------------------------------------
# Accepted paths.


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,H,D,T", [(1, 1, 64, 1), (3, 2, 128, 8), (5, 3, 256, 64), (40, 2, 64, 17)])
def test_accept_contiguous(dtype, B, H, D, T):
    """Bit-exact rows at the tails of ragged rows, none to all tokens, any order and repeats; every
    other slot as it was."""
    dev = cuda_or_skip()
    kvc = lib()
    gen = torch.Generator().manual_seed(B * 100 + T)
    cap = 100 + T
    k, v = randn((B, H, cap, D), 1, dev, dtype), randn((B, H, cap, D), 2, dev, dtype)
    kd, vd = randn((B, T, H, D), 3, dev, dtype), randn((B, T, H, D), 4, dev, dtype)
    lens = torch.randint(0, 101, (B, H), generator=gen).to(torch.int32).to(dev)
    n = torch.randint(0, T + 1, (B,), generator=gen).to(torch.int32).to(dev)
    n[0] = T
    path = torch.randint(0, T, (B, T), generator=gen).to(torch.int32).to(dev)
    want_k, want_v = k.clone(), v.clone()
    for b in range(B):
        for h in range(H):
            a, m = int(lens[b, h]), int(n[b])
            want_k[b, h, a:a + m] = kd[b, path[b, :m].long(), h]
            want_v[b, h, a:a + m] = vd[b, path[b, :m].long(), h]
    before = lens.clone()
    kvc.kvc_tree_accept(kvc.cache_view(k, v), lens, kvc.make_draft(kd, vd), path, n)
    assert kvc.kvc_device_status() == 0
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    assert torch.equal(lens, before + n[:, None])


def test_accept_refusals_leave_rows_as_they_were():
    """Out-of-range path entries, counts and lengths, and rows without room: recorded, nothing
    appended there, the others appended."""
    dev = cuda_or_skip()
    kvc = lib()
    B, H, D, T, cap = 3, 2, 64, 4, 20
    kd, vd = randn((B, T, H, D), 3, dev, torch.float32), randn((B, T, H, D), 4, dev, torch.float32)
    good = torch.tensor([[0, 1, 2, 3]] * B, dtype=torch.int32, device=dev)

    def run(lens, path, n, count=None):
        k, v = torch.zeros((B, H, cap, D), device=dev), torch.zeros((B, H, cap, D), device=dev)
        ln = torch.tensor(lens, dtype=torch.int32, device=dev)
        kvc.kvc_tree_accept(kvc.cache_view(k, v), ln, kvc.make_draft(kd, vd, count=count), path,
                            torch.tensor(n, dtype=torch.int32, device=dev))
        return kvc.kvc_device_status(), ln.tolist(), (k != 0).any(dim=3).sum(dim=2).tolist()

    ten = [[10, 10]] * B
    bad = good.clone()
    bad[1, 2] = T
    assert run(ten, bad, [3, 3, 2]) == (3, [[13, 13], [10, 10], [12, 12]], [[3, 3], [0, 0], [2, 2]])
    bad[1, 2] = -1
    assert run(ten, bad, [3, 3, 2])[1] == [[13, 13], [10, 10], [12, 12]]
    assert run(ten, bad, [3, 2, 2])[:2] == (0, [[13, 13], [12, 12], [12, 12]])   # not on the path
    assert run(ten, good, [5, -1, 4])[:2] == (5, [[10, 10], [10, 10], [14, 14]])
    assert run([[17, 16], [20, 0], [1, 2]], good, [4, 1, 1]) == \
        (1, [[17, 20], [20, 1], [2, 3]], [[0, 4], [0, 1], [1, 1]])
    # two kinds of refusal at once: whichever block records first (the codes keep the first)
    st, ln, rows = run([[17, 16], [20, 0], [21, -1]], good, [4, 1, 1])
    assert st in (1, 5) and ln == [[17, 20], [20, 1], [21, -1]] and rows == [[0, 4], [0, 1], [0, 0]]
    count = torch.tensor([4, 2, 0], dtype=torch.int32, device=dev)
    assert run(ten, good, [4, 3, 0], count)[:2] == (3, [[14, 14], [10, 10], [10, 10]])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bs", [1, 7, 16, 32])
def test_accept_paged(dtype, bs):
    """Pages opened as needed, ids from the top of the stack in sequence order, tables, lengths and
    rows as appending one by one would leave them."""
    dev = cuda_or_skip()
    kvc = lib()
    B, H, D, T = 6, 2, 64, 40
    lens = [0, 1, bs, 2 * bs - 1, 3 * bs, 5]
    mb = 50 if bs < 16 else 8
    kp, vp, table, nb, ln, score, free = paged_setup(dev, dtype, B, H, D, bs, lens, 8, spare=300)
    wide = torch.full((B, max(mb, table.shape[1])), -1, dtype=torch.int32, device=dev)
    wide[:, :table.shape[1]] = table
    table, score = wide, torch.full(wide.shape, 9.0, device=dev)
    top = torch.tensor([free.numel()], dtype=torch.int32, device=dev)
    kd, vd = randn((B, T, H, D), 3, dev, dtype), randn((B, T, H, D), 4, dev, dtype)
    gen = torch.Generator().manual_seed(bs)
    path = torch.stack([torch.randperm(T, generator=gen) for _ in range(B)]).to(torch.int32).to(dev)
    n = torch.tensor([T, 0, 1, 2, 17, 33], dtype=torch.int32, device=dev)
    want_k = [torch.cat([logical(kp, table, lens[b], bs, b), kd[b, path[b, :int(n[b])].long()].transpose(0, 1)], 1)
              for b in range(B)]
    want_v = [torch.cat([logical(vp, table, lens[b], bs, b), vd[b, path[b, :int(n[b])].long()].transpose(0, 1)], 1)
              for b in range(B)]
    ids = free.tolist()
    want_table = table.clone()
    opened = 0
    for b in range(B):
        old, new = -(-lens[b] // bs), -(-(lens[b] + int(n[b])) // bs)
        for i in range(old, new):
            want_table[b, i] = ids.pop()
            opened += 1
    got = kvc.kvc_tree_accept_paged(kvc.block_pool_view(kp, vp), kvc.page_table_view(table, nb, ln, score),
                                    kvc.free_pool_view(free, top), kvc.make_draft(kd, vd), path, n)
    assert kvc.kvc_device_status() == 0
    assert torch.equal(got, n) and int(top) == free.numel() - opened
    assert ln.tolist() == [a + int(m) for a, m in zip(lens, n)]
    assert nb.tolist() == [-(-int(x) // bs) for x in ln]
    assert torch.equal(table, want_table)
    for b in range(B):
        m = int(ln[b])
        assert torch.equal(logical(kp, table, m, bs, b), want_k[b])
        assert torch.equal(logical(vp, table, m, bs, b), want_v[b])
        old = -(-lens[b] // bs)
        assert bool((score[b, old:int(nb[b])] == 0).all()) and bool((score[b, :old] == 9).all())


def test_accept_paged_refusals():
    """A stack that cannot serve everyone (the sequences that fit are served, in order), a full
    table, lengths that disagree with the block count, a bad id: nothing else moves."""
    dev = cuda_or_skip()
    kvc = lib()
    B, H, D, bs, T = 4, 1, 64, 4, 8
    kd, vd = randn((B, T, H, D), 3, dev, torch.float32), randn((B, T, H, D), 4, dev, torch.float32)
    path = torch.arange(T, dtype=torch.int32, device=dev).repeat(B, 1)

    def run(lens, nbs, n, ids, top, mb=6):
        kp, vp = torch.zeros((H, 30, bs, D), device=dev), torch.zeros((H, 30, bs, D), device=dev)
        table = torch.arange(B * mb, dtype=torch.int32, device=dev).view(B, mb) % 20
        ln, nb = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (lens, nbs))
        fr = torch.tensor(ids, dtype=torch.int32, device=dev)
        tp = torch.tensor([top], dtype=torch.int32, device=dev)
        got = kvc.kvc_tree_accept_paged(
            kvc.block_pool_view(kp, vp), kvc.page_table_view(table, nb, ln, torch.zeros((B, mb), device=dev)),
            kvc.free_pool_view(fr, tp), kvc.make_draft(kd, vd), path,
            torch.tensor(n, dtype=torch.int32, device=dev))
        return kvc.kvc_device_status(), got.tolist(), ln.tolist(), nb.tolist(), int(tp)

    ids = [20, 21, 22, 23, 24]
    # needs 2, 2, 1, 1 with three ids: the second is skipped
    assert run([0, 0, 4, 3], [0, 0, 1, 1], [8, 8, 4, 2], ids, 3) == \
        (10, [8, 0, 4, 0], [8, 0, 8, 3], [2, 0, 2, 1], 0)
    assert run([0, 0, 4, 3], [0, 0, 1, 1], [1, 1, 1, 1], ids, 5)[:2] == (0, [1, 1, 1, 1])
    assert run([24, 23, 4, 0], [6, 6, 1, 0], [1, 1, 1, 0], ids, 5) == \
        (5, [0, 1, 1, 0], [24, 24, 5, 0], [6, 6, 2, 0], 4)
    assert run([4, 4, -1, 9], [2, 1, 0, 3], [1, 1, 1, 1], ids, 5)[:3] == \
        (5, [0, 1, 0, 1], [4, 5, -1, 10])
    st, got, ln, nb, top = run([0, 0, 0, 0], [0] * 4, [1, 1, 1, 1], [20, 21, 22, 77, 24], 5)
    assert st == 9 and got == [1, 0, 1, 1] and ln == [1, 0, 1, 1] and nb == [1, 0, 1, 1]
    assert run([0] * 4, [0] * 4, [1] * 4, ids, -3)[:2] == (10, [0, 0, 0, 0])


# --------------------------------------------------------------------------------------------
# A run of them together.


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verification_loop(dtype):
    """Draft, attend, accept, four times over a compressed cache and a paged copy of it: each
    step's attention is the definition over what was accepted so far, both caches agree, and the
    library's single-token decode reads the result."""
    dev = cuda_or_skip()
    kvc = lib()
    B, Hkv, G, D, T, bs = 2, 2, 4, 128, 10, 16
    n0 = [60, 33]
    cap = 160
    k, v = torch.full((B, Hkv, cap, D), NAN, device=dev, dtype=dtype), torch.full((B, Hkv, cap, D), NAN, device=dev, dtype=dtype)
    kp, vp, table, nb, ln, score, free = paged_setup(dev, dtype, B, Hkv, D, bs, n0, 8, spare=30)
    wide = torch.full((B, 12), -1, dtype=torch.int32, device=dev)
    wide[:, :table.shape[1]] = table
    table, score = wide, torch.zeros((B, 12), device=dev)
    top = torch.tensor([free.numel()], dtype=torch.int32, device=dev)
    pool, pt, fp = kvc.block_pool_view(kp, vp), kvc.page_table_view(table, nb, ln, score), kvc.free_pool_view(free, top)
    lens = torch.tensor([[n] * Hkv for n in n0], dtype=torch.int32, device=dev)
    for b in range(B):
        k[b, :, :n0[b]], v[b, :, :n0[b]] = logical(kp, table, n0[b], bs, b), logical(vp, table, n0[b], bs, b)
    gen = torch.Generator().manual_seed(1)
    for step in range(4):
        q = randn((B, T, Hkv * G, D), 10 + step, dev, dtype)
        kd, vd = randn((B, T, Hkv, D), 20 + step, dev, dtype), randn((B, T, Hkv, D), 30 + step, dev, dtype)
        mask = tree_masks(B, T, step).to(dev)
        draft = kvc.make_draft(kd, vd, mask=mask)
        out, lse = run_tree(kvc, q, k, v, kd, vd, lens, mask)
        verify(q, k, v, kd, vd, lens, mask, out, lse, what=f"step {step}")
        outp = kvc.kvc_decode_attn_tree_paged(q, pool, pt, draft, scale=1 / math.sqrt(D))
        # the accepted path: a leaf's ancestors
        path, n = torch.zeros((B, T), dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
        for b in range(B):
            leaf = int(torch.randint(0, T, (1,), generator=gen))
            anc = [i for i in range(T) if (int(mask[b, leaf]) >> i) & 1]
            path[b, :len(anc)] = torch.tensor(anc)
            n[b] = len(anc)
        path, n = path.to(dev), n.to(dev)
        kvc.kvc_tree_accept(kvc.cache_view(k, v), lens, draft, path, n)
        kvc.kvc_tree_accept_paged(pool, pt, fp, draft, path, n)
        assert torch.equal(lens[:, 0], ln) and torch.equal(lens[:, 1], ln)
        for b in range(B):
            m = int(ln[b])
            assert torch.equal(k[b, :, :m], logical(kp, table, m, bs, b))
            assert torch.equal(v[b, :, :m], logical(vp, table, m, bs, b))
        compare(outp, out.double(), 2.0 ** -6 * (1 + out.double().abs()) if dtype == torch.bfloat16
                else 1e-4 * (1 + out.double().abs()), "paged against contiguous")
    # a chain of one token whose row is in the cache already is the library's decode
    one = randn((B, 1, Hkv * G, D), 99, dev, dtype)
    k.nan_to_num_(0.0)
    v.nan_to_num_(0.0)
    dec = kvc.kvc_decode_attn(one[:, 0].contiguous(), k, v, scale=0.1, len=lens.view(-1))
    out, lse = run_tree(kvc, one, k, v, None, None, lens, None, scale=0.1)
    verify(one, k, v, None, None, lens, None, out, lse, scale=0.1)
    compare(dec, out[:, 0].double(), (2.0 ** -6 if dtype == torch.bfloat16 else 1e-4) *
            (1 + out[:, 0].double().abs()), "single-token decode")
    assert kvc.kvc_device_status() == 0
