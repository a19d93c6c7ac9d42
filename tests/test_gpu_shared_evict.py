"""Block eviction of sequences that hold pages together: forked, evicted, decoded and freed again, over bf16 and 8-bit
pages.  Every sequence attends to its own rows, and a page is free when its last holder has left it."""
import math
import random

import pytest
import torch

from q8_ref import attention

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_kvc_gb300 import kvc as k
    k.load()
    return k


class Serving:
    """A pool of NB pages, B sequences, and the rows that each of them is to hold, as the pages hold them."""

    def __init__(self, kvc, kind, B, NB, mb, H=2, G=2, D=64, bs=16):
        self.kvc, self.kind, self.B, self.NB, self.mb, self.H, self.G, self.D, self.bs = kvc, kind, B, NB, mb, H, G, D, bs
        dt = torch.uint8 if kind == "e4m3" else torch.bfloat16
        self.pools = [torch.zeros((H, NB, bs, D), dtype=dt, device=DEV) for _ in range(2)]
        self.scales = [torch.zeros((H, NB), device=DEV) for _ in range(2)]
        self.pool = kvc.block_pool_q8_view(*self.pools, *self.scales) if kind == "e4m3" else kvc.block_pool_view(*self.pools)
        self.table, self.nb, self.len = (torch.zeros(s, dtype=torch.int32, device=DEV) for s in ((B, mb), B, B))
        self.score = torch.zeros((B, mb), device=DEV)
        self.ids, self.top = torch.arange(NB, dtype=torch.int32, device=DEV), torch.tensor([NB], dtype=torch.int32, device=DEV)
        self.shares = torch.zeros(NB, dtype=torch.int32, device=DEV)
        self.pt, self.free = kvc.page_table_view(self.table, self.nb, self.len, self.score), kvc.free_pool_view(self.ids, self.top)
        self.scale = 1.0 / math.sqrt(D)

    def append(self, k, v):
        if self.kind == "e4m3":
            self.kvc.kvc_paged_append_q8(self.pool, self.pt, self.free, k, v)
        else:
            self.kvc.kvc_paged_append(self.pool, self.pt, self.free, k, v)

    def decode(self, q):
        logits, lse = torch.zeros((*q.shape[:2], self.mb * self.bs), device=DEV), torch.empty(q.shape[:2], device=DEV)
        call = self.kvc.kvc_decode_attn_paged_q8 if self.kind == "e4m3" else self.kvc.kvc_decode_attn_paged
        out = call(q, self.pool, self.pt, scale=self.scale, logits=logits, lse=lse)
        return out[0] if isinstance(out, tuple) else out, logits, lse

    def reorder(self, parent):
        self.kvc.kvc_pages_reorder(self.pool, self.pt, self.free, self.shares, torch.tensor(parent, dtype=torch.int32, device=DEV))

    def rows(self, b):
        """[2][H, n, D] in 64 bits."""
        n = int(self.len[b])
        t = self.table[b, : -(-n // self.bs)].long()
        if self.kind == "e4m3":
            return [(x[:, t].view(torch.float8_e4m3fn).double() * s[:, t].double()[..., None, None]).flatten(1, 2)[:, :n]
                    for x, s in zip(self.pools, self.scales)]
        return [x[:, t].double().flatten(1, 2)[:, :n] for x in self.pools]

    def consistent(self):
        """Counts are holders less one, and the rest of the pool is free, once."""
        held = {}
        for b in range(self.B):
            for x in self.table[b, :int(self.nb[b])].tolist():
                held[x] = held.get(x, 0) + 1
        free = self.ids[:int(self.top)].tolist()
        assert sorted(list(held) + free) == list(range(self.NB))
        assert self.shares.tolist() == [held.get(x, 1) - 1 for x in range(self.NB)]
        assert self.nb.tolist() == [-(-n // self.bs) for n in self.len.tolist()]


def new(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("seed", range(3))
def test_forked_sequences_are_evicted_and_decoded(kvc, kind, seed):
    B, mb, bs, budget = 4, 8, 16, 4
    s = Serving(kvc, kind, B, 60, mb)
    rng = random.Random(seed)
    released = torch.empty(B, dtype=torch.int32, device=DEV)
    for step in range(140):
        k, v = new(3 * step + 1000 * seed, B, s.H, s.D), new(3 * step + 1 + 1000 * seed, B, s.H, s.D)
        s.append(k, v)
        q = new(3 * step + 2 + 1000 * seed, B, s.H * s.G, s.D)
        out, logits, lse = s.decode(q)
        if step % 7 == 0:
            for b in range(B):
                kk, vv = s.rows(b)
                for h in range(s.H):
                    want, _, _, size = attention(q[b, h * s.G:(h + 1) * s.G].double(), kk[h], vv[h], s.scale)
                    # bf16 outputs 2^-8, and 2^-13 for weights of 16 bits and fp32 logits below 10
                    assert bool(((out[b, h * s.G:(h + 1) * s.G].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -13 * size).all())
        before = [(s.table[b, :int(s.nb[b])].tolist(), s.rows(b)) for b in range(B)]
        kvc.kvc_block_accumulate_evict(logits, lse, s.pt, s.free, block_size=bs, budget_blocks=budget, recent_blocks=1,
                                       released=released, shares=s.shares)
        s.consistent()
        for b, r in enumerate(released.tolist()):        # what stays is what was there, without the released page
            ids, rows = before[b]
            if r >= 0:
                ids = ids[:r] + ids[r + 1:]
                rows = [torch.cat([x[:, :r * bs], x[:, (r + 1) * bs:]], dim=1) for x in rows]
            assert s.table[b, :int(s.nb[b])].tolist() == ids
            assert all(torch.equal(x, y) for x, y in zip(s.rows(b), rows))
        if step % 11 == 10:
            s.reorder([rng.randrange(B) for _ in range(B)])
            s.consistent()
    s.reorder([-1] * B)
    assert int(s.top) == 60 and not bool(s.shares.any()) and kvc.kvc_device_status() == 0


@pytest.mark.parametrize("B", [2, 3, 64, 500])
def test_a_page_that_all_leave_at_once(kvc, B):
    """Sequences forked from one, whose oldest page leaves all of them in one call: it is freed once.  Some keep it."""
    s = Serving(kvc, "bf16", B, 3 * B + 3, 4, H=1, G=1)      # (33 rows are three pages each, before they are shared)
    for step in range(33):
        x = new(step, B, 1, s.D)
        s.append(x, x)
        if step == 0:
            s.reorder([0] * B)
    s.reorder([0] * B)
    s.consistent()
    page = int(s.table[0, 0])
    assert int(s.shares[page]) == B - 1 and int(s.top) == s.NB - 2 - B
    _, logits, lse = s.decode(new(99, B, 1, s.D))
    s.score.zero_()
    s.score[:, 1] = 1e6
    s.score[: B // 3, :2] = torch.tensor([1e6, 0.0], device=DEV)           # these leave their second page
    kvc.kvc_block_accumulate_evict(logits, lse, s.pt, s.free, block_size=16, budget_blocks=2, recent_blocks=1, shares=s.shares)
    s.consistent()
    assert int(s.shares[page]) == max(B // 3 - 1, 0)
    assert (page in s.ids[:int(s.top)].tolist()) == (B // 3 == 0)
    assert kvc.kvc_device_status() == 0


def test_an_id_outside_the_pool_is_kept(kvc):
    s = Serving(kvc, "bf16", 2, 10, 4, H=1, G=1)
    for step in range(33):
        x = new(step, 2, 1, s.D)
        s.append(x, x)
    _, logits, lse = s.decode(new(99, 2, 1, s.D))
    s.score.zero_()
    s.score[:, 1] = 1e6
    released = torch.full((2,), 7, dtype=torch.int32, device=DEV)
    for bad in (10, -1):
        s.table[0, 0] = bad
        before = [x.clone() for x in (s.table[0], s.nb[0], s.len[0])]
        top, nb = int(s.top), int(s.nb[1])
        kvc.kvc_block_accumulate_evict(logits, lse, s.pt, s.free, block_size=16, budget_blocks=1, recent_blocks=1, released=released,
                                       shares=s.shares)
        assert kvc.kvc_device_status() == 9
        assert all(torch.equal(x, y) for x, y in zip(before, (s.table[0], s.nb[0], s.len[0]))) and int(released[0]) == -1
        assert int(released[1]) >= 0 and int(s.nb[1]) == nb - 1 and int(s.top) == top + 1
    assert not bool(s.shares.any())


def test_pages_of_one_holder_are_evicted_as_before(kvc):
    """Counts of zero: the same tables, scores and stack as the call without them."""
    runs = []
    for shared in (False, True):
        s = Serving(kvc, "bf16", 1, 20, 6, H=1, G=2)
        for step in range(90):
            x = new(step, 1, 1, s.D)
            s.append(x, x)
            _, logits, lse = s.decode(new(500 + step, 1, 2, s.D))
            kvc.kvc_block_accumulate_evict(logits, lse, s.pt, s.free, block_size=16, budget_blocks=3, recent_blocks=1,
                                           **({"shares": s.shares} if shared else {}))
        runs.append([x.clone() for x in (s.table[:, :3], s.nb, s.len, s.score[:, :3], s.ids, s.top)])
    assert all(torch.equal(x, y) for x, y in zip(*runs)) and kvc.kvc_device_status() == 0


def test_captured_and_on_another_stream(kvc):
    s = Serving(kvc, "bf16", 3, 30, 6, H=1, G=1)
    for step in range(40):
        x = new(step, 3, 1, s.D)
        s.append(x, x)
    s.reorder([0, 0, 0])
    s.consistent()
    _, logits, lse = s.decode(new(99, 3, 1, s.D))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kvc.kvc_block_accumulate_evict(logits, lse, s.pt, s.free, block_size=16, budget_blocks=2, recent_blocks=1, shares=s.shares, stream=side)
    side.synchronize()
    s.consistent()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.kvc_block_accumulate_evict(logits, lse, s.pt, s.free, block_size=16, budget_blocks=1, recent_blocks=1, shares=s.shares)
    graph.replay()
    s.consistent()
    assert s.nb.tolist() == [1, 1, 1] and kvc.kvc_device_status() == 0
