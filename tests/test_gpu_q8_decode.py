"""Attention over 8-bit pages against the definition in 64 bits."""
import math

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


class Case:
    """Pages of random numbers whose scales differ by 2^+-spread, behind shuffled tables; what lies
    behind a length, and every page in no table, is NaN."""

    def __init__(self, kvc, lens, Hq, H, D, bs, dt, *, seed=0, spread=3, power=True, max_blocks=None, qsize=1.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        cpu = torch.Generator().manual_seed(seed)
        B = len(lens)
        nb = [(n + bs - 1) // bs for n in lens]
        mb = max_blocks or max(1, max(nb))
        NB = sum(nb) + 3
        table = torch.full((B, mb), -1, dtype=torch.int32)
        perm, at = torch.randperm(NB, generator=cpu).to(torch.int32), 0
        self.k, self.v = (torch.full((H, NB, bs, D), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2))
        for b, n in enumerate(lens):
            table[b, :nb[b]] = perm[at:at + nb[b]]
            at += nb[b]
            for pool in (self.k, self.v):
                x = (torch.randn((H, nb[b] * bs, D), generator=g, device=DEV) * 100).clamp(-448, 448)
                x = x.to(torch.float8_e4m3fn).view(torch.uint8)
                x[:, n:] = 0x7F
                pool[:, table[b, :nb[b]].long().to(DEV)] = x.view(H, nb[b], bs, D)
        e = torch.rand((2, H, NB), generator=g, device=DEV) * 2 * spread - spread
        e = torch.exp2(e.round() if power else e)
        self.ks, self.vs = e[0] / 256, e[1] / 100
        self.table, self.lens, self.dt = table.to(DEV), lens, dt
        self.len = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.nb = torch.tensor(nb, dtype=torch.int32, device=DEV)
        self.q = (torch.randn((B, Hq, D), generator=g, device=DEV) * qsize).to(dt)
        self.scale = 1.0 / math.sqrt(D)
        self.kvc, self.bs, self.H, self.D, self.G, self.mb = kvc, bs, H, D, Hq // H, mb
        self.pool = kvc.block_pool_q8_view(self.k, self.v, self.ks, self.vs)
        self.score = torch.zeros((B, mb), device=DEV)
        self.pt = kvc.page_table_view(self.table, self.nb, self.len, self.score)

    def rows(self, b, h):
        n = self.lens[b]
        t = self.table[b, : (n + self.bs - 1) // self.bs].long()
        return ((x[h, t].view(torch.float8_e4m3fn).double() * s[h, t].double()[:, None, None]).flatten(0, 1)[:n]
                for x, s in ((self.k, self.ks), (self.v, self.vs)))

    def call(self, **kw):
        B, Hq = self.q.shape[:2]
        self.logits = torch.full((B, Hq, self.mb * self.bs + 3), 7.5, device=DEV)
        self.lse = torch.empty((B, Hq), device=DEV)
        self.out = self.kvc.kvc_decode_attn_paged_q8(self.q, self.pool, self.pt, scale=self.scale, logits=self.logits,
                                                     lse=self.lse, **kw)
        return self.out

    def check(self, which=None):
        """Errors, per element:  a logit x = scale * ks * q . k8 takes D products with at most (D + 8)
        roundings of 2^-23 (the product's sums are cut, not rounded), fp32 queries are cut to 22 bits of
        the row's largest element, and its factors and log2(e) are four roundings; a weight is off by twice
        the largest logit error (its own and its maximum's), by the last place of a difference of two
        such logits and of ex2 (2^-21 in all), and by its rounding: 2^-11 to fp16 for bf16 queries,
        2^-22 as two terms; a sum over n slots adds n / 16 + 16 cut partial sums and merges them.
        The output adds half a step of its type."""
        G, n_max = self.G, max(self.lens)
        f32 = self.dt == torch.float32
        for b in range(len(self.lens)) if which is None else which:
            n = self.lens[b]
            for h in range(self.H):
                k, v = self.rows(b, h)
                q = self.q[b, h * G:(h + 1) * G].double()
                want, lse, x, size = attention(q, k, v, self.scale)
                got = self.out[b, h * G:(h + 1) * G].double()
                got_lse = self.lse[b, h * G:(h + 1) * G].double()
                lg = None if self.logits is None else self.logits[b, h * G:(h + 1) * G]
                assert lg is None or bool((lg[:, n:] == 7.5).all())
                if n == 0:
                    assert bool((got == 0).all()) and bool((got_lse == -math.inf).all())
                    continue
                dx = abs(self.scale) * (self.D + 8) * 2.0 ** -23 * (q.abs() @ k.abs().T) + x.abs() * 2.0 ** -22
                if f32:
                    dx = dx + abs(self.scale) * 2.0 ** -22 * q.abs().amax(dim=1, keepdim=True) * k.abs().sum(dim=1)
                assert lg is None or bool(((lg[:, :n].double() - x).abs() <= dx).all())
                p = torch.softmax(x, dim=1)
                # a logit counts by its weight: those of weight 2^-40 move nothing
                big = (dx * (p > 2.0 ** -40)).amax(dim=1, keepdim=True)
                rel = 2 * big + 2.0 ** -21 + (2.0 ** -22 if f32 else 2.0 ** -11) + (n / 16 + 32) * 2.0 ** -23
                tol = rel * size + torch.finfo(self.dt).eps / 2 * want.abs() + 2.0 ** -30 * v.abs().amax()
                assert bool(((got - want).abs() <= tol).all()), (b, h, float(((got - want).abs() / tol).max()))
                tol = big[:, 0] + 2.0 ** -21 + (n_max / 16 + 32) * 2.0 ** -23 + lse.abs() * 2.0 ** -22
                assert bool(((got_lse - lse).abs() <= tol).all())
        assert self.kvc.kvc_device_status() == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,Hq,H,D,bs", [
    ([1], 1, 1, 64, 16), ([0, 1, 15, 16, 17], 4, 2, 64, 16), ([31, 32, 33, 0, 127, 128, 129], 8, 1, 128, 32),
    ([200, 3, 0], 6, 1, 256, 16), ([100, 131], 24, 2, 128, 64), ([1, 2, 3, 400], 32, 1, 64, 48),
    ([77, 600], 40, 2, 256, 32), ([513], 5, 5, 128, 16), ([16, 16, 16, 16], 17, 1, 128, 16)])
def test_against_the_definition(kvc, dt, lens, Hq, H, D, bs):
    c = Case(kvc, lens, Hq, H, D, bs, dt, seed=1)
    c.call()
    c.check()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_long_row_over_all_ranges(kvc, dt):
    c = Case(kvc, [20011], 8, 1, 128, 32, dt, seed=2)
    c.call()
    c.check()
    first = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.call()
        assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


@pytest.mark.parametrize("D,Hq,H", [(64, 4, 2), (128, 16, 1), (256, 6, 1)])
def test_ragged_batches(kvc, D, Hq, H):
    c = Case(kvc, [4000, 0, 17, 1, 2222, 640, 0, 3], Hq, H, D, 16, torch.bfloat16, seed=3)
    c.call()
    c.check()


@pytest.mark.parametrize("lens,Hq,H,bs", [
    ([4000, 0, 17, 1, 2222, 640, 0, 3], 9, 1, 16), ([1500, 3, 700], 32, 2, 32), ([9001], 31, 1, 64),
    ([(53 * b) % 401 for b in range(90)], 48, 4, 16)])
def test_groups_of_nine_to_sixteen_in_fp32(kvc, lens, Hq, H, bs):
    """Row tiles of 16 heads, whose queries and weights are two terms each."""
    c = Case(kvc, lens, Hq, H, 128, bs, torch.float32, seed=9)
    c.call()
    c.check(which=list(range(0, len(lens), 1 + len(lens) // 30)))


def test_more_row_tiles_than_ranges(kvc):
    """Thousands of rows: split ones are noted by the range they begin in."""
    lens = [(37 * b) % 301 for b in range(700)]
    c = Case(kvc, lens, 8, 4, 64, 16, torch.bfloat16, seed=4)
    c.call()
    c.check(which=list(range(0, 700, 23)))


def test_short_rows_in_thousands(kvc):
    """Tables of so few slots that no row is split."""
    lens = [(11 * b) % 65 for b in range(1500)]
    c = Case(kvc, lens, 4, 2, 64, 16, torch.bfloat16, seed=5)
    c.call()
    c.check(which=list(range(0, 1500, 41)) + [1499])


def test_batches_without_any_slots(kvc):
    for n, mb in ((1, 1), (5, 100), (400, 100)):
        c = Case(kvc, [0] * n, 8, 2, 128, 16, torch.bfloat16, seed=6, max_blocks=mb)
        c.call()
        c.check()


def test_row_tiles_of_one_slot_in_thousands(kvc):
    c = Case(kvc, [1 + b % 3 for b in range(6000)], 1, 1, 64, 16, torch.float32, seed=6)
    c.call()
    c.check(which=list(range(0, 6000, 307)) + [5999])


def test_pools_beyond_32_bits_of_bytes(kvc):
    """Pages at the end of a pool of more than 2^32 bytes, in every call that reads or writes them."""
    H, NB, bs, D, B = 2, 140000, 64, 256, 2
    assert H * NB * bs * D > 2 ** 32
    k, v = (torch.zeros((H, NB, bs, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = torch.zeros((H, NB), device=DEV), torch.zeros((H, NB), device=DEV)
    table = torch.zeros((B, 4), dtype=torch.int32, device=DEV)
    nb, lens = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    ids = torch.arange(NB, dtype=torch.int32, device=DEV)       # the last pages are popped first
    top = torch.tensor([NB], dtype=torch.int32, device=DEV)
    pool, free = kvc.block_pool_q8_view(k, v, ks, vs), kvc.free_pool_view(ids, top)
    pt = kvc.page_table_view(table, nb, lens, torch.zeros((B, 4), device=DEV))
    x = torch.randn((300, H, D), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(torch.bfloat16)
    cu = torch.tensor([0, 200, 300], dtype=torch.int32, device=DEV)
    kvc.kvc_paged_append_q8(pool, pt, free, x, -x, cu=cu)
    assert table[0].tolist() == [NB - 1, NB - 2, NB - 3, NB - 4]
    q = torch.randn((B, 4, D), generator=torch.Generator(device=DEV).manual_seed(2), device=DEV).to(torch.bfloat16)
    want = kvc.kvc_decode_attn_paged_q8(q, pool, pt, scale=0.05)
    for b, n in enumerate([200, 100]):
        t = table[b, : (n + bs - 1) // bs].long()
        for h in range(H):
            kk, vv = ((p[h, t].view(torch.float8_e4m3fn).double() * s[h, t].double()[:, None, None]).flatten(0, 1)[:n]
                      for p, s in ((k, ks), (v, vs)))
            # half a step of 4 significant bits, and of the smallest step of a page
            rows = x[int(cu[b]):int(cu[b]) + n, h].double()
            assert bool(((kk - rows).abs() <= 2.0 ** -4 * rows.abs() + 2.0 ** -17 * rows.abs().max()).all())
            assert torch.equal(vv, -kk)
            ref, _, _, size = attention(q[b, 2 * h:2 * h + 2].double(), kk, vv, 0.05)
            # bf16 outputs 2^-8, weights 2^-11, and 2^-14 for fp32 logits below 10
            assert bool(((want[b, 2 * h:2 * h + 2].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.0 ** -14) * size).all())
    shares = torch.zeros(NB, dtype=torch.int32, device=DEV)
    kvc.kvc_pages_reorder(pool, pt, free, shares, torch.tensor([1, 1], dtype=torch.int32, device=DEV))
    out = kvc.kvc_decode_attn_paged_q8(q, pool, pt, scale=0.05)
    assert torch.equal(out[1], want[1])
    same = kvc.kvc_decode_attn_paged_q8(q[1:].expand(2, 4, D).contiguous(), pool, pt, scale=0.05)
    assert torch.equal(same[0], same[1])
    kvc.kvc_pages_compact(pool, pt, free, shares=shares)
    assert torch.equal(kvc.kvc_decode_attn_paged_q8(q, pool, pt, scale=0.05), out)
    assert int(table[:, :2].max()) < 4 and kvc.kvc_device_status() == 0


def test_tables_of_the_largest_capacity(kvc):
    """2^30 slots a sequence: the units of all row tiles pass 32 bits, whatever the lengths."""
    c = Case(kvc, [700, 0, 33, 5000], 16, 8, 64, 1024, torch.bfloat16, seed=6, max_blocks=2 ** 20)
    c.lse, c.logits = torch.empty((4, 16), device=DEV), None
    c.out = kvc.kvc_decode_attn_paged_q8(c.q, c.pool, c.pt, scale=c.scale, lse=c.lse)
    c.check()


def test_a_workspace_too_small_is_refused(kvc):
    c = Case(kvc, [40], 4, 2, 64, 16, torch.bfloat16, seed=6)
    n = kvc.kvc_decode_attn_paged_q8_workspace_bytes(1, 4, 2, 64, kvc.KVC_BF16)
    c.call(ws=torch.empty(n + 256, dtype=torch.uint8, device=DEV))
    with pytest.raises(kvc.KvcError):
        c.call(ws=torch.empty(n - 1, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_scales_of_any_size(kvc, dt):
    """Pages whose scales are no powers of two and differ by 2^40: keys, then values."""
    c = Case(kvc, [300, 90], 4, 2, 64, 16, dt, seed=6, power=False)
    c.vs *= torch.exp2(torch.randint(-20, 20, c.vs.shape, device=DEV).float())
    c.call()
    c.check()
    c.vs.fill_(2.0 ** -120)
    c.vs[:, c.table[0, 3].long()] = 2.0 ** 100
    c.call()
    c.check()


def test_a_page_of_small_values_and_large_weights(kvc):
    """The weight lies on pages whose values are 2^-60 of the others': they still count in full."""
    c = Case(kvc, [64], 1, 1, 64, 16, torch.float32, seed=7)
    c.vs.fill_(1.0)
    t = c.table[0].long()
    c.vs[:, t[1]] = 2.0 ** -60
    # the slots of page 1 get a logit of 100, the others 0
    c.ks.fill_(1.0 / 256)
    c.k[:, t] = torch.where(c.k[:, t] == 0x7F, c.k[:, t], torch.zeros_like(c.k[:, t]))
    c.k[:, t[1]] = torch.full((16, 64), 100.0, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    c.q.fill_(1.0)
    c.scale = 4.0
    out = c.call()
    _, v = c.rows(0, 0)
    x = torch.tensor([100.0 / 256 * 64 * 4], dtype=torch.float64).item()
    rest = math.exp(-x)
    want = (v[16:32].sum(dim=0) + rest * (v[:16].sum(dim=0) + v[32:].sum(dim=0))) / (16 + 48 * rest)
    # e^-100 is 2^-144: the other pages' part is below the last place of 2^-60
    assert rest < 2.0 ** -100
    assert bool(((out[0, 0].double() - want).abs() <= 2.0 ** -18 * v[16:32].abs().mean(dim=0) + 1e-30).all())


@pytest.mark.parametrize("size", [2.0 ** -60, 1.0, 2.0 ** 20, 2.0 ** 60])
def test_queries_of_any_size(kvc, size):
    c = Case(kvc, [200, 50], 4, 2, 128, 32, torch.bfloat16, seed=8, qsize=size)
    c.scale = 1.0 / (math.sqrt(128) * size)
    c.call()
    c.check()


@pytest.mark.parametrize("scale", [0.0, -0.3, 300.0])
def test_scales_of_the_logits(kvc, scale):
    """Zero: all slots alike; negative; so large that one slot takes all."""
    c = Case(kvc, [150, 20], 4, 2, 64, 16, torch.float32, seed=9)
    c.scale = scale
    c.call()
    c.check()


def test_zero_queries_and_zero_pages(kvc):
    c = Case(kvc, [40, 33], 4, 2, 64, 16, torch.bfloat16, seed=10)
    c.q[0, 1] = 0
    c.k[:, c.table[1, 0].long()] = 0
    c.v[:, c.table[1, 1].long()] = 0
    c.vs[:, c.table[1, 1].long()] = 2.0 ** -120
    c.call()
    c.check()


def test_nan_reaches_the_rows_that_see_it(kvc):
    c = Case(kvc, [40, 33], 4, 2, 64, 16, torch.bfloat16, seed=11)
    t = c.table[0].long()
    c.v[1, t[1], 3, 10] = 0x7F
    out = c.call()
    bad = torch.zeros(out.shape, dtype=torch.bool, device=DEV)
    bad[0, 2:4, 10] = True
    assert torch.equal(out.isnan(), bad)
    c.k[0, t[0], 5, 0] = 0xFF
    out = c.call()
    bad[0, :2] = True
    assert torch.equal(out.isnan(), bad) and bool(c.lse[0, :2].isnan().all())


def test_lengths_and_ids_outside_their_range(kvc):
    c = Case(kvc, [40, 48, 20], 4, 2, 64, 16, torch.bfloat16, seed=12)
    want = c.call().clone()
    c.len[2] = -5
    out = c.call()
    assert kvc.kvc_device_status() == 5
    assert torch.equal(out[:2], want[:2]) and bool((out[2] == 0).all())
    c.len.copy_(torch.tensor([40, 1000, 20]))    # clamped to the table: 48
    out = c.call()
    assert kvc.kvc_device_status() == 5 and torch.equal(out, want)
    c.len.copy_(torch.tensor([40, 48, 20]))
    c.table[0, 1] = 10 ** 7
    out = c.call()
    assert kvc.kvc_device_status() == 9 and torch.equal(out[1:], want[1:])


def test_tables_longer_than_a_window_of_ids(kvc):
    """Page ids are read 32 at a time: rows that begin and end inside such a window."""
    c = Case(kvc, [16 * 33 + 5, 16 * 64, 16 * 31, 16 * 100 + 1], 2, 1, 64, 16, torch.bfloat16, seed=13, max_blocks=150)
    c.call()
    c.check()


def test_captured_and_on_another_stream(kvc):
    c = Case(kvc, [300, 0, 45], 8, 2, 128, 32, torch.bfloat16, seed=14)
    want = c.call().clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.kvc.kvc_decode_attn_paged_q8(c.q, c.pool, c.pt, scale=c.scale, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out, ws = torch.zeros_like(c.q), kvc.decode_q8_workspace(3, 8, 2, 128, torch.bfloat16, DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.kvc_decode_attn_paged_q8(c.q, c.pool, c.pt, scale=c.scale, out=out, ws=ws)
    for n in (300, 17, 289):                     # the lengths live on the device
        c.len[0] = n
        graph.replay()
        assert torch.equal(out, c.call())
