"""Pages shared between sequences and pools made dense, against a model of lists."""
import random

import pytest
import torch

from q8_ref import Pages

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = ("k", "v", "table", "n_blocks", "len", "score", "shares", "ids", "top", "pos")


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_kvc_gb300 import kvc as k
    k.load()
    return k


class Cache:
    """A pool in which every row is told apart, tables of shuffled ids, counts and positions."""

    def __init__(self, kvc, lens, H=2, D=64, bs=16, spare=20, max_blocks=12, seed=0, kind="bf16"):
        g = torch.Generator().manual_seed(seed)
        self.kvc, self.bs, self.kind, B = kvc, bs, kind, len(lens)
        nb = [(n + bs - 1) // bs for n in lens]
        NB = sum(nb) + spare
        perm = torch.randperm(NB, generator=g).to(torch.int32)
        if kind == "e4m3":
            self.k, self.v = (torch.randint(0, 256, (H, NB, bs, D), generator=g, dtype=torch.uint8).to(DEV) for _ in range(2))
            self.ks, self.vs = (torch.rand((H, NB), generator=g).to(DEV) for _ in range(2))
            self.pool = kvc.block_pool_q8_view(self.k, self.v, self.ks, self.vs)
        else:
            dt = torch.bfloat16 if kind == "bf16" else torch.float32
            self.k, self.v = (torch.randn((H, NB, bs, D), generator=g).to(dt).to(DEV) for _ in range(2))
            self.ks = self.vs = None
            self.pool = kvc.block_pool_view(self.k, self.v)
        table = torch.full((B, max_blocks), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(nb):
            table[b, :n] = perm[at:at + n]
            at += n
        ids = torch.full((NB,), -9, dtype=torch.int32)
        ids[:NB - at] = perm[at:]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
        for name, x in dict(table=table, ids=ids, top=i32([NB - at]), n_blocks=i32(nb), len=i32(lens),
                            score=torch.rand((B, max_blocks), generator=g), shares=torch.zeros(NB, dtype=torch.int32),
                            pos=torch.arange(NB * bs, dtype=torch.int32).view(NB, bs)).items():
            setattr(self, name, x.to(DEV))
        self.pt = kvc.page_table_view(self.table, self.n_blocks, self.len, self.score)
        self.free = kvc.free_pool_view(self.ids, self.top)
        self.model = Pages(table, self.n_blocks, self.len, self.score, self.ids, self.top, bs, self.shares)
        self.rows = [self.read(b) for b in range(B)]         # what every sequence holds

    def read(self, b):
        n = int(self.len[b])
        t = self.table[b, : (n + self.bs - 1) // self.bs].long()
        out = [x[:, t].flatten(1, 2)[:, :n].clone() for x in (self.k, self.v)] + [self.pos[t].flatten()[:n].clone()]
        if self.ks is not None:
            out += [x[:, t].repeat_interleave(self.bs, dim=1)[:, :n].clone() for x in (self.ks, self.vs)]
        return out

    def reorder(self, parent, **kw):
        par = torch.tensor(parent, dtype=torch.int32, device=DEV)
        self.kvc.kvc_pages_reorder(self.pool, self.pt, self.free, self.shares, par, pos=self.pos, **kw)
        self.model.reorder(parent)
        empty = [x[:, :0] if x.dim() > 1 else x[:0] for x in self.rows[0]]
        self.rows = [self.rows[p] if p >= 0 else empty for p in parent]

    def append(self, seed):
        """One token more for every sequence that holds any."""
        B, (H, _, _, D) = len(self.rows), self.k.shape
        g = torch.Generator().manual_seed(seed)
        k, v = (torch.randn((B, H, D), generator=g).to(self.k.dtype).to(DEV) for _ in range(2))
        t = torch.tensor([10 ** 6 + seed], device=DEV)
        self.kvc.kvc_paged_append(self.pool, self.pt, self.free, k, v, t=t, pos=self.pos)
        # ids that several sequences pop in one such call depend on timing: the model takes them over
        for b in range(B):
            if self.model.len[b] % self.bs == 0:
                lb = self.model.n_blocks[b]
                self.model.table[b][lb], self.model.score[b][lb] = int(self.table[b, lb]), 0.0
                self.model.n_blocks[b] += 1
            self.model.len[b] += 1
            r = self.rows[b]
            self.rows[b] = [torch.cat([r[0], k[b][:, None]], dim=1), torch.cat([r[1], v[b][:, None]], dim=1),
                            torch.cat([r[2], t.to(torch.int32)])]
        self.model.top = int(self.top)
        self.model.ids = self.ids.tolist()

    def check(self):
        self.model.same_as(self.table, self.n_blocks, self.len, self.score, self.ids, self.top, self.shares)
        for b, want in enumerate(self.rows):
            for x, y in zip(self.read(b), want):
                assert torch.equal(x, y)
        held = {}
        for b in range(len(self.rows)):
            for i, x in enumerate(self.table[b, :int(self.n_blocks[b])].tolist()):
                held[x] = held.get(x, 0) + 1
        free = self.ids[:int(self.top)].tolist()
        assert sorted(list(held) + free) == list(range(self.k.shape[1]))
        shares = self.shares.tolist()
        assert all(shares[x] == n - 1 for x, n in held.items()) and all(shares[x] == 0 for x in free)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("H,D,bs,lens,parent", [
    (1, 64, 16, [0], [0]), (1, 64, 16, [17], [-1]), (2, 128, 32, [40, 0, 0, 0], [0, 0, 0, 0]),
    (2, 64, 16, [5, 16, 33, 64], [3, 2, 1, 0]), (3, 256, 16, [31, 32, 1], [1, 1, 1]),
    (2, 64, 64, [63, 64, 65, 130], [-1, 0, -1, 3]), (1, 128, 16, [20, 20, 20, 20], [1, 1, 2, 2]),
    (2, 64, 16, [0, 18], [1, 0]), (2, 64, 16, [18, 18], [0, 1])])
def test_one_reorder(kvc, kind, H, D, bs, lens, parent):
    c = Cache(kvc, lens, H, D, bs, kind=kind)
    c.reorder(parent)
    assert kvc.kvc_device_status() == 0
    c.check()


def test_shared_pages_outlive_their_holders(kvc):
    c = Cache(kvc, [50, 0, 0, 0])
    c.reorder([0, 0, 0, -1])
    c.check()
    assert int(c.shares.max()) == 2
    c.reorder([-1, 1, 2, -1])                    # the parent is done, its children go on
    c.check()
    c.reorder([-1, -1, 2, 2])
    c.check()
    c.reorder([-1] * 4)
    c.check()
    assert int(c.top) == c.k.shape[1] and kvc.kvc_device_status() == 0


@pytest.mark.parametrize("seed", range(4))
def test_beams_that_grow_and_are_reordered(kvc, seed):
    """Appends, reorders and compactions in turn, as a beam search makes them."""
    rng = random.Random(seed)
    c = Cache(kvc, [rng.randint(1, 40) for _ in range(6)], bs=16, spare=60, seed=seed, kind="bf16")
    ws = kvc.pages_workspace(6, 12, c.k.shape[1], DEV)
    for step in range(25):
        c.append(1000 * seed + step)
        if step % 2:
            c.reorder([rng.randrange(6) for _ in range(6)], ws=ws)
        if step % 7 == 6:
            compact(kvc, c, ws=ws)
        c.check()
    assert kvc.kvc_device_status() == 0


@pytest.mark.parametrize("B,mb", [(1, 3000), (3, 700), (1500, 4), (8192, 1)])
def test_tables_of_many_shapes(kvc, B, mb):
    rng = random.Random(B)
    c = Cache(kvc, [rng.randint(0, min(mb * 16, 4000 if B > 3 else 10 ** 6)) for _ in range(B)], H=1, bs=16,
              spare=B + 5, max_blocks=mb)
    c.reorder([rng.randrange(-1, B) for _ in range(B)])
    assert kvc.kvc_device_status() == 0
    c.model.same_as(c.table, c.n_blocks, c.len, c.score, c.ids, c.top, c.shares)
    for b in rng.sample(range(B), min(B, 20)):
        for x, y in zip(c.read(b), c.rows[b]):
            assert torch.equal(x, y)


def state(c):
    return {n: getattr(c, n).clone() for n in NAMES}


def unchanged(c, before):
    for n in NAMES:
        assert torch.equal(getattr(c, n), before[n]), n


@pytest.mark.parametrize("code,change", [
    (3, lambda c, par: par.__setitem__(1, 4)), (3, lambda c, par: par.__setitem__(0, -2)),
    (5, lambda c, par: c.len.__setitem__(2, -1)), (5, lambda c, par: c.len.__setitem__(2, 10 ** 6)),
    (5, lambda c, par: c.n_blocks.__setitem__(1, 1)), (9, lambda c, par: c.table.__setitem__((0, 1), -1)),
    (9, lambda c, par: c.table.__setitem__((0, 0), 10 ** 7)), (12, lambda c, par: c.shares.__setitem__(int(c.table[0, 1]), 1)),
    (10, lambda c, par: c.top.fill_(-1)), (10, lambda c, par: c.top.fill_(10 ** 6)),
    (10, lambda c, par: c.top.fill_(0)), (9, lambda c, par: c.ids.__setitem__(int(c.top) - 1, -4))])
def test_reorder_refusals_change_nothing(kvc, code, change):
    c = Cache(kvc, [20, 33, 7, 7])
    par = torch.tensor([0, 0, 2, 0], dtype=torch.int32, device=DEV)
    if code == 10 or "ids" in change.__code__.co_names:
        par[2] = 0                               # (no page is freed that a copy could take)
        c.len[1], c.n_blocks[1], c.len[2], c.n_blocks[2], c.len[3], c.n_blocks[3] = 0, 0, 0, 0, 0, 0
    change(c, par)
    before = state(c)
    kvc.kvc_pages_reorder(c.pool, c.pt, c.free, c.shares, par, pos=c.pos)
    assert kvc.kvc_device_status() == code
    unchanged(c, before)


def _far(c, par, code):
    if code == 10:
        par[2] = 0
        c.len[1:], c.n_blocks[1:] = 0, 0


@pytest.mark.parametrize("code,change", [
    (3, lambda c, par: par.__setitem__(1, 4)), (5, lambda c, par: c.len.__setitem__(2, 10 ** 6)),
    (5, lambda c, par: c.n_blocks.__setitem__(1, 1)), (9, lambda c, par: c.table.__setitem__((0, 1), -1)),
    (12, lambda c, par: c.shares.__setitem__(int(c.table[0, 1]), 1)), (10, lambda c, par: c.top.fill_(-1)),
    (10, lambda c, par: c.top.fill_(0)), (9, lambda c, par: c.table.__setitem__((3, 0), int(c.table[2, 0])))])
@pytest.mark.parametrize("mb", [2048, 2049])
def test_reorder_refusals_of_large_tables(kvc, mb, code, change):
    """Tables of 256 and 260 runs of 32 entries, of one block and of a cluster."""
    c = Cache(kvc, [20, 33, 16, 16], max_blocks=mb)
    par = torch.tensor([0, 0, -1, -1], dtype=torch.int32, device=DEV)
    _far(c, par, code)
    change(c, par)
    before = state(c)
    kvc.kvc_pages_reorder(c.pool, c.pt, c.free, c.shares, par, pos=c.pos)
    assert kvc.kvc_device_status() == code
    unchanged(c, before)


@pytest.mark.parametrize("mb", [12, 2100])
def test_reorders_in_turn_with_few_free_pages(kvc, mb):
    """The same reorders over short tables (one block) and long ones (a cluster), the stack almost empty."""
    rng = random.Random(7)
    c = Cache(kvc, [rng.randint(0, 40) for _ in range(5)], bs=16, spare=9, max_blocks=mb, kind="e4m3")
    for step in range(20):
        c.reorder([rng.choice([-1, 0, 1, 2, 3, 4, b]) for b in range(5)])
        c.check()
    assert kvc.kvc_device_status() == 0


@pytest.mark.parametrize("NB", [32767, 32768, 33900, 34300])
def test_reorder_in_a_pool_that_just_fits_shared_memory(kvc, NB):
    c = Cache(kvc, [40, 17, 0, 90], H=1, D=64, spare=NB - 11)
    assert c.k.shape[1] == NB
    c.reorder([3, 0, 0, -1])
    c.check()
    c.reorder([2, 1, 1, 0])
    c.check()
    assert kvc.kvc_device_status() == 0


def test_pages_listed_more_often_than_counted(kvc):
    c = Cache(kvc, [32, 32])
    c.table[1, 0] = c.table[0, 0]
    before = state(c)
    kvc.kvc_pages_reorder(c.pool, c.pt, c.free, c.shares, torch.tensor([-1, -1], dtype=torch.int32, device=DEV))
    assert kvc.kvc_device_status() == 9
    unchanged(c, before)


def test_a_stack_without_room(kvc):
    c = Cache(kvc, [32, 32], spare=3)
    small = kvc.free_pool_view(c.ids[:4].clone(), c.top)
    before = state(c)
    kvc.kvc_pages_reorder(c.pool, c.pt, small, c.shares, torch.tensor([0, -1], dtype=torch.int32, device=DEV))
    assert kvc.kvc_device_status() == 11
    unchanged(c, before)


def test_freed_pages_serve_the_copies_of_the_same_call(kvc):
    """An empty stack: the page that one beam gives up is the page that another one needs."""
    c = Cache(kvc, [20, 21, 22], spare=0)
    c.reorder([0, 0, 2])
    assert kvc.kvc_device_status() == 0
    c.check()


# ------------------------------------------------------------------------------------------
def compact(kvc, c, **kw):
    NB, m = c.k.shape[1], c.model
    remap = kvc.kvc_pages_compact(c.pool, c.pt, c.free, shares=c.shares, pos=c.pos, **kw).tolist()
    free = set(m.ids[:m.top])
    live = NB - m.top
    want = [-1 if x in free else x for x in range(NB)]
    holes = [x for x in range(live) if x in free]
    for x, to in zip([x for x in range(live, NB) if x not in free], holes):
        want[x] = to
    assert remap == want
    m.table = [[want[x] for x in r[:n]] + r[n:] for r, n in zip(m.table, m.n_blocks)]
    shares = [0] * NB
    for x in range(NB):
        if want[x] >= 0:
            shares[want[x]] = m.shares[x]
    m.shares = shares
    m.ids[:m.top] = [NB - 1 - i for i in range(m.top)]


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("H,D,bs,lens,spare", [
    (1, 64, 16, [0], 1), (1, 64, 16, [16], 0), (2, 128, 32, [40, 0, 95, 33], 9), (3, 256, 16, [100, 20], 40),
    (2, 64, 64, [300, 1], 3), (1, 64, 16, [150] * 12, 100)])
def test_one_compaction(kvc, kind, H, D, bs, lens, spare):
    c = Cache(kvc, lens, H, D, bs, spare, kind=kind)
    compact(kvc, c)
    assert kvc.kvc_device_status() == 0
    c.check()
    used = {x for r, n in zip(c.model.table, c.model.n_blocks) for x in r[:n]}
    assert used == set(range(len(used)))
    compact(kvc, c)                              # a dense pool stays as it is
    c.check()


def test_compaction_of_shared_pages(kvc):
    c = Cache(kvc, [50, 30, 0, 0], spare=30)
    c.reorder([0, 0, 0, -1])
    compact(kvc, c)
    c.check()
    c.reorder([-1, 1, 1, 2])
    c.check()


def test_live_pages_outside_the_tables_move_too(kvc):
    c = Cache(kvc, [40, 20], spare=30)
    kept = c.ids[int(c.top) - 5:int(c.top)].clone().long()         # taken by someone else
    c.top -= 5
    rows = c.k[:, kept].clone()
    remap = kvc.kvc_pages_compact(c.pool, c.pt, c.free)
    assert kvc.kvc_device_status() == 0
    assert bool((remap[kept] >= 0).all()) and torch.equal(c.k[:, remap[kept].long()], rows)


def test_a_large_pool(kvc):
    lens = [16 * 500] * 40
    c = Cache(kvc, lens, H=1, spare=13777, max_blocks=500)
    compact(kvc, c)
    assert kvc.kvc_device_status() == 0
    c.model.same_as(c.table, c.n_blocks, c.len, c.score, c.ids, c.top, c.shares)
    for b in (0, 17, 39):
        for x, y in zip(c.read(b), c.rows[b]):
            assert torch.equal(x, y)


def test_the_largest_pool(kvc):
    """2^20 pages, one in a thousand live and anywhere."""
    NB, n = 2 ** 20, 1000
    g = torch.Generator().manual_seed(1)
    perm = torch.randperm(NB, generator=g).to(torch.int32)
    k, v = (torch.zeros((1, NB, 16, 64), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = torch.zeros((1, NB), device=DEV), torch.zeros((1, NB), device=DEV)
    table = perm[:n].view(4, 250).to(DEV)
    ks[0, table.long()] = torch.arange(n, device=DEV).float().view(4, 250)
    ids = torch.zeros(NB, dtype=torch.int32)
    ids[:NB - n] = perm[n:]
    ids, top = ids.to(DEV), torch.tensor([NB - n], dtype=torch.int32, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    pt = kvc.page_table_view(table, i32([250] * 4), i32([4000] * 4), torch.zeros((4, 250), device=DEV))
    remap = kvc.kvc_pages_compact(kvc.block_pool_q8_view(k, v, ks, vs), pt, kvc.free_pool_view(ids, top))
    assert kvc.kvc_device_status() == 0
    assert sorted(table.flatten().tolist()) == list(range(n)) and int((remap >= 0).sum()) == n
    assert torch.equal(ks[0, table.long()], torch.arange(n, device=DEV).float().view(4, 250))
    assert torch.equal(ids[:NB - n], torch.arange(NB - 1, n - 1, -1, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("code,change", [
    (10, lambda c: c.top.fill_(-1)), (10, lambda c: c.top.fill_(10 ** 6)), (9, lambda c: c.ids.__setitem__(0, -1)),
    (9, lambda c: c.ids.__setitem__(0, 10 ** 6)), (9, lambda c: c.ids.__setitem__(0, int(c.ids[1]))),
    (9, lambda c: c.ids.__setitem__(2, int(c.table[0, 0]))), (9, lambda c: c.table.__setitem__((1, 0), -5)),
    (5, lambda c: c.n_blocks.__setitem__(0, 13)), (5, lambda c: c.n_blocks.__setitem__(1, -1))])
def test_compaction_refusals_change_nothing(kvc, code, change):
    c = Cache(kvc, [40, 20], spare=30)
    change(c)
    before = state(c)
    remap = torch.full((c.k.shape[1],), 77, dtype=torch.int32, device=DEV)
    kvc.kvc_pages_compact(c.pool, c.pt, c.free, shares=c.shares, pos=c.pos, remap=remap)
    assert kvc.kvc_device_status() == code
    unchanged(c, before)
    assert bool((remap == 77).all())


def test_captured_and_on_another_stream(kvc):
    c = Cache(kvc, [50, 20, 0, 5], spare=30)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.reorder([0, 0, 1, 3], stream=side)
    side.synchronize()
    c.check()
    par = torch.zeros(4, dtype=torch.int32, device=DEV)
    ws = kvc.pages_workspace(4, 12, c.k.shape[1], DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.kvc_pages_reorder(c.pool, c.pt, c.free, c.shares, par, pos=c.pos, ws=ws)
    for parent in ([0, 1, 2, 2], [3, 2, 1, 0], [1, 1, -1, 1]):
        par.copy_(torch.tensor(parent))
        graph.replay()
        c.model.reorder(parent)
        c.rows = [c.rows[p] if p >= 0 else [x[:, :0] if x.dim() > 1 else x[:0] for x in c.rows[0]] for p in parent]
        c.check()
