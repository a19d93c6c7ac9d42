"""Rows into 8-bit pages: numbers, scales, page tables and refusals against a model that takes the rows
one page after the other in 64 bits.  All of it is compared for equality."""
import numpy as np
import pytest
import torch

from q8_ref import Pages, numbers, quantise_into

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_kvc_gb300 import kvc as k
    k.load()
    return k


class Cache:
    """A pool, tables and a free stack of shuffled ids; sequences begin with lens[b] rows of random numbers."""

    def __init__(self, kvc, lens, H=2, D=64, bs=16, spare=20, max_blocks=12, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.kvc, self.bs, B = kvc, bs, len(lens)
        nb = [(n + bs - 1) // bs for n in lens]
        NB = sum(nb) + spare
        perm = torch.randperm(NB, generator=g).to(torch.int32)
        self.k, self.v = (torch.randint(0, 256, (H, NB, bs, D), generator=g, dtype=torch.uint8) for _ in range(2))
        self.k[self.k & 127 == 127] = 0          # (no NaN)
        self.v[self.v & 127 == 127] = 0
        self.ks, self.vs = (torch.exp2(torch.randint(-6, 3, (H, NB), generator=g).float()) for _ in range(2))
        table = torch.full((B, max_blocks), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(nb):
            table[b, :n] = perm[at:at + n]
            at += n
        ids = torch.full((NB,), -9, dtype=torch.int32)
        ids[:NB - at] = perm[at:]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
        for name, x in dict(k=self.k, v=self.v, ks=self.ks, vs=self.vs, table=table, ids=ids, top=i32([NB - at]),
                            n_blocks=i32(nb), len=i32(lens), score=torch.rand((B, max_blocks), generator=g)).items():
            setattr(self, name, x.to(DEV))
        self.pool = kvc.block_pool_q8_view(self.k, self.v, self.ks, self.vs)
        self.pt = kvc.page_table_view(self.table, self.n_blocks, self.len, self.score)
        self.free = kvc.free_pool_view(self.ids, self.top)
        self.model = Pages(table, self.n_blocks, self.len, self.score, self.ids, self.top, bs)
        self.mk, self.mv = numbers(self.k), numbers(self.v)
        self.mks, self.mvs = self.ks.double().cpu().numpy(), self.vs.double().cpu().numpy()

    def append(self, counts, k_new, v_new, **kw):
        """counts: rows of each sequence (the model's); k_new, v_new on the GPU."""
        cu = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
        self.kvc.kvc_paged_append_q8(self.pool, self.pt, self.free, k_new, v_new, cu=cu, **kw)
        self.expect(counts, k_new, v_new)

    def expect(self, counts, k_new, v_new, rows_of=None):
        first = np.concatenate([[0], np.cumsum(counts)]) if rows_of is None else rows_of
        kx, vx = (x.double().cpu().numpy() for x in (k_new, v_new))
        for b, page, held, at, n in self.model.append(counts):
            r = int(first[b]) + at
            quantise_into(self.mk, self.mks, page, held, kx[r:r + n])
            quantise_into(self.mv, self.mvs, page, held, vx[r:r + n])

    def check(self):
        self.model.same_as(self.table, self.n_blocks, self.len, self.score, self.ids, self.top)
        for got, want in ((self.k, self.mk), (self.v, self.mv)):
            np.testing.assert_array_equal(numbers(got), want)
        np.testing.assert_array_equal(self.ks.double().cpu().numpy(), self.mks)
        np.testing.assert_array_equal(self.vs.double().cpu().numpy(), self.mvs)


def rows(seed, dt, n, H, D, spread=8.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((n, H, D), generator=g, device=DEV)
    return (x * torch.exp2(torch.rand((n, 1, 1), generator=g, device=DEV) * spread - spread / 2)).to(dt)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,D,bs,lens,counts", [
    (1, 64, 16, [0], [1]), (2, 64, 16, [0, 15, 16, 17, 31], [1, 1, 1, 1, 1]), (3, 128, 32, [0, 5, 32], [100, 27, 3]),
    (1, 256, 64, [70, 0], [129, 64]), (2, 128, 16, [3, 0, 9, 40], [0, 50, 0, 8]), (2, 256, 48, [47, 48], [2, 97]),
    (1, 128, 128, [100], [300]), (5, 64, 32, [1] * 7, [33, 0, 31, 32, 1, 2, 64])])
def test_rows_of_ragged_sequences(kvc, dt, H, D, bs, lens, counts):
    c = Cache(kvc, lens, H, D, bs)
    n = sum(counts)
    appended = torch.full((len(lens),), -1, dtype=torch.int32, device=DEV)
    c.append(counts, rows(1, dt, n, H, D), rows(2, dt, n, H, D), appended=appended)
    c.check()
    assert appended.tolist() == counts and kvc.kvc_device_status() == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,D,bs", [(3, 64, 16), (2, 64, 32), (2, 64, 64), (2, 128, 16), (1, 128, 48), (2, 256, 16),
                                    (1, 256, 32), (1, 256, 128)])
def test_prompts_in_pages_of_every_size(kvc, dt, H, D, bs):
    """One to eight warps hold a page, or take it in parts; pages begun before, and infinities."""
    lens, counts = [3, 0, bs, 2 * bs - 1], [5 * bs + 7, 1, 3 * bs, 90]
    c = Cache(kvc, lens, H, D, bs)
    n = sum(counts)
    k, v = rows(50, dt, n, H, D) * 3, rows(51, dt, n, H, D)
    k[2, 0, 5], v[counts[0], H - 1, D - 1] = float("-inf"), float("inf")
    c.append(counts, k, v)
    c.check()
    assert kvc.kvc_device_status() == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,D", [(3, 64), (2, 128), (1, 256)])
def test_steps_of_uneven_counts(kvc, dt, H, D):
    """A few rows a sequence, groups of lanes side by side: some with raised scales, infinities, NaN or no rows."""
    lens, counts = [3, 16, 31, 0, 7, 40], [1, 0, 9, 2, 5, 3]
    c = Cache(kvc, lens, H, D, 16)
    n = sum(counts)
    for step in range(3):
        k, v = rows(60 + step, dt, n, H, D), rows(70 + step, dt, n, H, D)
        k[0], v[4, H - 1] = k[0] * 2.0 ** 12, v[4, H - 1] * 2.0 ** 20
        k[2, 0, 5], k[13, H - 1, 1], v[19, 0, 0] = float("inf"), float("nan"), float("-inf")
        c.append(counts, k, v)
        c.check()
    assert kvc.kvc_device_status() == 0


def test_single_tokens_without_offsets(kvc):
    """Rows that raise a page's scale bring the ones there to it; many steps over page borders."""
    c = Cache(kvc, [0, 7, 16, 30], 2, 128, 16)
    for i in range(40):
        k, v = rows(100 + i, torch.bfloat16, 4, 2, 128), rows(200 + i, torch.bfloat16, 4, 2, 128)
        kvc.kvc_paged_append_q8(c.pool, c.pt, c.free, k, v)
        c.expect([1] * 4, k, v)
    c.check()
    assert kvc.kvc_device_status() == 0


def test_one_by_one_is_at_once_but_for_the_smallest(kvc):
    """Sizes within 2^8 of the page's largest: no number falls below 2^-6, and the pages are the same."""
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((32, 2, 64), generator=g, device=DEV)
    x = (x.sign() * torch.exp2(torch.rand(x.shape, generator=g, device=DEV) * 8)).to(torch.bfloat16)
    a, b = Cache(kvc, [0], 2, 64, 32), Cache(kvc, [0], 2, 64, 32)
    a.append([32], x, -x)
    for i in range(32):
        kvc.kvc_paged_append_q8(b.pool, b.pt, b.free, x[i:i + 1], -x[i:i + 1])
    page = int(a.table[0, 0])
    assert page == int(b.table[0, 0])
    assert torch.equal(a.k[:, page], b.k[:, page]) and torch.equal(a.v[:, page], b.v[:, page])
    assert torch.equal(a.ks, b.ks) and torch.equal(a.vs, b.vs)


def test_scale_at_its_borders(kvc):
    """Largest sizes of exactly 448 s, the next float above, zeros, the smallest and the largest floats."""
    c = Cache(kvc, [0] * 8, 1, 64, 16)
    x = torch.zeros((8, 1, 64), device=DEV)
    up = torch.nextafter(torch.tensor(448.0), torch.tensor(1e9)).item()
    for i, big in enumerate([448.0, up, 0.0, 1e-45, 3.4e38, 2.0 ** -112, 7.0, -1792.0]):
        x[i, 0, 5] = big
        x[i, 0, 6] = big / 3
    kvc.kvc_paged_append_q8(c.pool, c.pt, c.free, x, -x)
    c.expect([1] * 8, x, -x)
    c.check()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_non_finite_elements(kvc, dt):
    c = Cache(kvc, [0, 5], 2, 64, 16)
    k, v = rows(4, dt, 24, 2, 64), rows(5, dt, 24, 2, 64)
    k[1, 0, 3], k[2, 1, 60], v[20, 0, 0], v[21, 1, 1] = (float(x) for x in ("inf", "-inf", "nan", "inf"))
    v[3] = float("nan")
    c.append([14, 10], k, v)
    c.check()


def test_scales_of_another_kind_are_continued(kvc):
    """Partly filled pages whose scales are no powers of two: kept where they are large, else raised."""
    c = Cache(kvc, [5, 9, 3], 2, 64, 16)
    for s, m in ((c.ks, c.mks), (c.vs, c.mvs)):
        s.copy_(torch.rand(s.shape, device=DEV) * 0.02 + 0.001)
        m[:] = s.double().cpu().numpy()
    c.append([4, 2, 1], rows(6, torch.float32, 7, 2, 64), rows(7, torch.float32, 7, 2, 64))
    c.check()


def test_strided_rows(kvc):
    """Keys and values as slices of one projection's output, and head-major rows."""
    H, D = 3, 64
    qkv = rows(8, torch.bfloat16, 20, 4 * H, D)
    c = Cache(kvc, [10, 0], H, D, 16)
    c.append([13, 7], qkv[:, 2 * H:3 * H], qkv[:, 3 * H:])
    turned = rows(9, torch.bfloat16, H, 20, D).transpose(0, 1)
    c.append([13, 7], turned, turned)
    c.check()


def test_more_sequences_than_one_block_scans(kvc):
    B = 2500
    c = Cache(kvc, [(7 * b) % 33 for b in range(B)], 1, 64, 16, spare=6000, max_blocks=6)
    counts = [(5 * b) % 40 for b in range(B)]
    k = rows(10, torch.bfloat16, sum(counts), 1, 64)
    c.append(counts, k, k.flip(0))
    c.check()
    one = rows(11, torch.bfloat16, B, 1, 64)
    kvc.kvc_paged_append_q8(c.pool, c.pt, c.free, one, one)
    c.expect([1] * B, one, one)
    c.check()


def refused(kvc, c, before, code):
    assert kvc.kvc_device_status() == code
    for name, x in before.items():
        assert torch.equal(getattr(c, name), x), name


def snapshot(c):
    return {n: getattr(c, n).clone() for n in ("k", "v", "ks", "vs", "table", "ids", "top", "n_blocks", "len", "score")}


@pytest.mark.parametrize("cu", [[0, 3, 2, 5], [0, 2, 4, 6], [-1, 1, 2, 3], [0, 2 ** 31 - 1, -5, 3]])
def test_bad_offsets_append_nothing(kvc, cu):
    c = Cache(kvc, [0, 5, 16])
    before, x = snapshot(c), rows(12, torch.bfloat16, 5, 2, 64)
    got = torch.full((3,), -1, dtype=torch.int32, device=DEV)
    kvc.kvc_paged_append_q8(c.pool, c.pt, c.free, x, x, cu=torch.tensor(cu, dtype=torch.int32, device=DEV), appended=got)
    refused(kvc, c, before, 5)
    assert got.tolist() == [0, 0, 0]


def test_sequences_that_cannot_be_served(kvc):
    """Lengths that disagree, a full table, a bad id of the partly filled page: left alone, the others served."""
    c = Cache(kvc, [16, 20, 12 * 16 - 1, 5, 3], spare=30)
    c.n_blocks[1] += 1
    c.table[3, 0] = 10 ** 6
    x = rows(13, torch.bfloat16, 12, 2, 64)
    keep = snapshot(c)
    cu = torch.tensor([0, 2, 4, 6, 8, 12], dtype=torch.int32, device=DEV)
    got = torch.full((5,), -1, dtype=torch.int32, device=DEV)
    kvc.kvc_paged_append_q8(c.pool, c.pt, c.free, x, x, cu=cu, appended=got)
    assert kvc.kvc_device_status() in (5, 9) and got.tolist() == [2, 0, 0, 0, 4]
    c.expect([2, 0, 0, 0, 4], x, x, rows_of=cu.tolist())
    c.model.n_blocks[1] += 1
    assert c.len.tolist() == c.model.len and int(c.top) == c.model.top
    assert c.table[3].tolist() == keep["table"][3].tolist()
    np.testing.assert_array_equal(numbers(c.k), c.mk)
    np.testing.assert_array_equal(c.vs.double().cpu().numpy(), c.mvs)


def test_an_empty_stack_serves_whom_it_can(kvc):
    c = Cache(kvc, [16, 16, 15, 16], spare=3)
    x = rows(14, torch.bfloat16, 70, 2, 64)
    cu = torch.tensor([0, 17, 52, 53, 70], dtype=torch.int32, device=DEV)     # 2, 3, 0, 2 pages
    got = torch.full((4,), -1, dtype=torch.int32, device=DEV)
    kvc.kvc_paged_append_q8(c.pool, c.pt, c.free, x, x, cu=cu, appended=got)
    assert kvc.kvc_device_status() == 10 and got.tolist() == [17, 0, 1, 0]
    c.expect([17, 0, 1, 0], x, x, rows_of=cu.tolist())
    c.check()


def test_bad_ids_leave_the_stack(kvc):
    c = Cache(kvc, [16, 16, 16], spare=6)
    good = c.ids[:6].tolist()
    c.ids[4] = -3                                # the second page popped
    x = rows(15, torch.bfloat16, 18, 2, 64)
    cu = torch.tensor([0, 17, 18, 18], dtype=torch.int32, device=DEV)         # two pages, then one
    got = torch.full((3,), -1, dtype=torch.int32, device=DEV)
    kvc.kvc_paged_append_q8(c.pool, c.pt, c.free, x, x, cu=cu, appended=got)
    assert kvc.kvc_device_status() == 9 and got.tolist() == [0, 1, 0]
    assert int(c.top) == 4 and c.ids[:4].tolist() == good[:4]
    assert c.table[1, 1].item() == good[5] and c.len.tolist() == [16, 17, 16]


def test_a_stack_top_outside_the_stack(kvc):
    c = Cache(kvc, [16])
    c.top.fill_(10 ** 6)
    before, x = snapshot(c), rows(16, torch.bfloat16, 1, 2, 64)
    kvc.kvc_paged_append_q8(c.pool, c.pt, c.free, x, x)
    refused(kvc, c, before, 10)


def test_no_rows_at_all(kvc):
    c = Cache(kvc, [3, 16])
    before, x = snapshot(c), torch.empty((0, 2, 64), device=DEV)
    kvc.kvc_paged_append_q8(c.pool, c.pt, c.free, x, x, cu=torch.zeros(3, dtype=torch.int32, device=DEV))
    refused(kvc, c, before, 0)


def test_captured_and_on_another_stream(kvc):
    c = Cache(kvc, [0, 9], spare=30)
    x = rows(17, torch.bfloat16, 2, 2, 64)
    ws = kvc.append_q8_workspace(2, 2, 16, DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kvc.kvc_paged_append_q8(c.pool, c.pt, c.free, x, x, stream=side)
    side.synchronize()
    c.expect([1, 1], x, x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.kvc_paged_append_q8(c.pool, c.pt, c.free, x, x, ws=ws)
    for i in range(20):
        x.copy_(rows(300 + i, torch.bfloat16, 2, 2, 64))
        graph.replay()
        c.expect([1, 1], x, x)
    c.check()
