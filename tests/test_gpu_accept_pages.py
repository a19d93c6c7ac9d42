"""GPU: what kvc_tree_accept_paged refuses, against a model that takes the sequences one by one: a
sequence is appended whole or not at all, and what it does not use stays on the free stack."""
import pytest
import torch

from gpu_helpers import cuda_or_skip, lib
from tree_ref import randn

pytestmark = pytest.mark.gpu
BAD_LENGTH, BAD_BLOCK, POOL_EMPTY = 5, 9, 10


class Pages:
    """A pool, page tables and a free stack on the device, with the same state as lists."""

    def __init__(self, dev, bs, n_pool, lens, tables, ids, mb, H=2, D=64, T=8):
        self.bs, self.n_pool, self.H, self.T = bs, n_pool, H, T
        B = len(lens)
        self.lens, self.tables, self.ids = list(lens), [list(t) for t in tables], list(ids)
        self.kp, self.vp = (randn((H, n_pool, bs, D), s, dev, torch.float32) for s in (1, 2))
        self.kd, self.vd = (randn((B, T, H, D), s, dev, torch.float32) for s in (3, 4))
        self.table = torch.full((B, mb), 123456789, dtype=torch.int32, device=dev)
        for b, t in enumerate(self.tables):
            if t:
                self.table[b, :len(t)] = torch.tensor(t, dtype=torch.int32)
        self.score = torch.full((B, mb), 9.0, device=dev)
        self.ln = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.nb = torch.tensor([len(t) for t in tables], dtype=torch.int32, device=dev)
        self.free = torch.tensor(ids, dtype=torch.int32, device=dev)
        self.top = torch.tensor([len(ids)], dtype=torch.int32, device=dev)
        gen = torch.Generator().manual_seed(B)
        self.path = torch.randint(0, T, (B, T), generator=gen).to(torch.int32)
        self.wk, self.wv = self.kp.cpu().clone(), self.vp.cpu().clone()

    def model(self, n):
        """Appends n[b] tokens to every sequence in turn; returns accepted and the codes recorded."""
        accepted, codes = [], set()
        kd, vd = self.kd.cpu(), self.vd.cpu()
        for b, want in enumerate(n):
            t, ln = self.tables[b], self.lens[b]
            need = -(-(ln + want) // self.bs) - len(t) if want else 0
            take = self.ids[len(self.ids) - need:] if need else []
            sound = [i for i in take if 0 <= i < self.n_pool]
            got = 0
            if want and ln % self.bs and not 0 <= t[-1] < self.n_pool:
                codes.add(BAD_BLOCK)
            elif need > len(self.ids):
                codes.add(POOL_EMPTY)
            elif len(sound) < need:                # the bad ids leave the stack, the others stay
                codes.add(BAD_BLOCK)
                self.ids[len(self.ids) - need:] = sound
            else:
                got = want
                if need:
                    del self.ids[-need:]
                t += take[::-1]
                for i in range(want):
                    slot, src = ln + i, int(self.path[b, i])
                    blk, off = t[slot // self.bs], slot % self.bs
                    self.wk[:, blk, off], self.wv[:, blk, off] = kd[b, src], vd[b, src]
                self.lens[b] += want
            accepted.append(got)
        return accepted, codes

    def check(self, kvc, n):
        dev = self.kp.device
        old = [len(t) for t in self.tables]
        want, codes = self.model(n)
        got = kvc.kvc_tree_accept_paged(
            kvc.block_pool_view(self.kp, self.vp),
            kvc.page_table_view(self.table, self.nb, self.ln, self.score),
            kvc.free_pool_view(self.free, self.top), kvc.make_draft(self.kd, self.vd),
            self.path.to(dev), torch.tensor(n, dtype=torch.int32, device=dev))
        status = kvc.kvc_device_status()
        assert got.tolist() == want
        assert status in codes if codes else status == 0
        assert self.ln.tolist() == self.lens and self.nb.tolist() == [len(t) for t in self.tables]
        assert int(self.top) == len(self.ids) and self.free[:len(self.ids)].tolist() == self.ids
        table, score = self.table.tolist(), self.score.tolist()
        for b, t in enumerate(self.tables):
            assert table[b] == t + [123456789] * (self.table.shape[1] - len(t))
            assert score[b][:len(t)] == [9.0] * old[b] + [0.0] * (len(t) - old[b])
        assert torch.equal(self.kp.cpu(), self.wk) and torch.equal(self.vp.cpu(), self.wv)
        return want, codes


@pytest.mark.parametrize("bad", [40, -1, 2 ** 31 - 1, -2 ** 31])
def test_a_bad_last_page_refuses_its_sequence(bad):
    """The partly filled page that the first accepted token would go to is outside the pool: the
    sequence is left as it was.  A full page is not written, so whatever stands there does not
    matter, nor does it where nothing is accepted."""
    dev = cuda_or_skip()
    p = Pages(dev, 4, 40, [5, 6, 4, 3, 7], [[0, bad], [1, 2], [bad], [bad], [3, bad]], [20, 21, 22, 23], 5)
    want, codes = p.check(lib(), [2, 3, 2, 0, 8])
    assert want == [0, 3, 2, 0, 0] and codes == {BAD_BLOCK}


def test_bad_ids_leave_the_stack_and_the_others_stay():
    """A sequence that would take an id outside the pool is refused; the id is dropped, the good ones
    taken with it serve the sequences behind, in the stack's order."""
    dev = cuda_or_skip()
    none = [[] for _ in range(4)]
    # the first needs two blocks and finds one: the good one stays for the second
    p = Pages(dev, 4, 40, [0] * 4, none, [20, 21, 22, 77, 24], 4)
    assert p.check(lib(), [5, 3, 8, 0]) == ([0, 3, 8, 0], {BAD_BLOCK}) and p.ids == [20]
    # with the last good id kept, the second is served; the third finds an empty stack
    p = Pages(dev, 4, 40, [0] * 4, none, [20, -5], 4)
    assert p.check(lib(), [8, 4, 1, 0]) == ([0, 4, 0, 0], {BAD_BLOCK, POOL_EMPTY}) and p.ids == []
    # nothing but bad ids; a sequence that needs no block is appended all the same
    p = Pages(dev, 4, 40, [0, 5, 0, 0], [[], [30, 31], [], []], [99, -1, 40], 4)
    assert p.check(lib(), [5, 3, 4, 4]) == ([0, 3, 0, 0], {BAD_BLOCK, POOL_EMPTY})
    # too few ids for the first, a bad one for the second, good ones for the others
    p = Pages(dev, 2, 40, [0] * 4, none, [20, 21, 40], 4)
    assert p.check(lib(), [8, 3, 2, 1]) == ([0, 0, 2, 1], {BAD_BLOCK, POOL_EMPTY}) and p.ids == []


@pytest.mark.parametrize("B,bad,short", [(1, 1, 0), (33, 0, 1), (33, 3, 0), (33, 6, 1), (1300, 0, 0),
                                         (1300, 9, 0), (1300, 0, 1), (1300, 40, 1)])
def test_many_sequences_with_bad_ids_and_a_short_stack(B, bad, short):
    """More sequences than the kernel takes at once, bad ids anywhere on the stack, a stack that cannot
    serve everyone, bad last pages: as one sequence after another."""
    dev = cuda_or_skip()
    gen = torch.Generator().manual_seed(B * 100 + bad * 2 + short)

    def rand(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=gen))

    bs = 3
    lens = [rand(0, 6) for _ in range(B)]
    n = [rand(0, 8) for _ in range(B)]
    held = sum(-(-x // bs) for x in lens)
    need = sum(-(-(x + m) // bs) - -(-x // bs) for x, m in zip(lens, n))
    spare = need // 2 if short else need + 5
    n_pool = held + spare
    order = torch.randperm(n_pool, generator=gen).tolist()
    tables = []
    for x in lens:
        tables.append([order.pop() for _ in range(-(-x // bs))])
    ids = order
    for _ in range(min(bad, len(ids))):
        ids[rand(0, len(ids) - 1)] = n_pool + rand(0, 1000)
    if bad > 3:
        for b in range(0, B, 7):
            if tables[b]:
                tables[b][-1] = -rand(1, 1000)
    p = Pages(dev, bs, n_pool, lens, tables, ids, 6, H=1)
    want, codes = p.check(lib(), n)
    assert sum(want) > 0 or B == 1
    assert bad or short or (want == n and not codes)
