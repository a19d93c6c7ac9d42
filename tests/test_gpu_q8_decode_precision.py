"""Attention over 8-bit pages where few bits would show: logits of any size, rows of one heavy slot and
a hundred thousand light ones, weights that are all rounded alike, warps that walk a thousand steps."""
import math

import pytest
import torch

from q8_ref import attention

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_kvc_gb300 import kvc as k
    k.load()
    return k


class Cache:
    """k, v [B, H, n, D]: e4m3 numbers; ks, vs [B, H, pages of bs]: their scales."""

    def __init__(self, kvc, k, v, ks, vs, bs, seed=0):
        B, H, n, D = k.shape
        per = -(-n // bs)
        pad = per * bs - n
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32).to(DEV)
        at = self.table.flatten().long()
        self.pools, self.scales = [], []
        for x, s in ((k, ks), (v, vs)):
            x = torch.nn.functional.pad(x, (0, 0, 0, pad), value=float("nan")).to(torch.float8_e4m3fn).view(torch.uint8)
            pool = torch.empty((H, B * per, bs, D), dtype=torch.uint8, device=DEV)
            pool[:, at] = x.view(B, H, per, bs, D).transpose(0, 1).reshape(H, B * per, bs, D)
            scale = torch.empty((H, B * per), device=DEV)
            scale[:, at] = s.transpose(0, 1).reshape(H, B * per)
            self.pools.append(pool)
            self.scales.append(scale)
        self.len = torch.full((B,), n, dtype=torch.int32, device=DEV)
        self.nb = torch.full((B,), per, dtype=torch.int32, device=DEV)
        self.score = torch.zeros((B, per), device=DEV)
        self.pool = kvc.block_pool_q8_view(*self.pools, *self.scales)
        self.pt = kvc.page_table_view(self.table, self.nb, self.len, self.score)
        # the rows as the definition has them
        self.k, self.v = ((x.double() * s.double().repeat_interleave(bs, dim=2)[:, :, :n, None]) for x, s in ((k, ks), (v, vs)))


def decode(kvc, c, q, scale):
    lse = torch.empty(q.shape[:2], device=DEV)
    out = kvc.kvc_decode_attn_paged_q8(q, c.pool, c.pt, scale=scale, lse=lse)
    assert kvc.kvc_device_status() == 0
    return out, lse


def positive(shape, seed):
    """e4m3 numbers in [1, 2)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(8, 16, shape, generator=g, device=DEV) / 8.0


def cut_sums(n, rows):
    """Sums that a number of an output passes through.  Each product of 16 slots adds once or twice (the
    weights are two terms) in the warp that has them; a row alone is dealt out evenly to 8 warps or more of every
    SM, several rows at most one warp each; then come at most 24 parts of a block, 8 sets of parts of
    several blocks, and the 152 / 8 parts of such a set."""
    warps = 8 * torch.cuda.get_device_properties(0).multi_processor_count / rows
    return 2 * (n / 16 / max(1.0, warps) + 2) + 24 + 8 + 19


def step(dt):
    """The rounding of an output."""
    return torch.finfo(dt).eps / 2


# ------------------------------------------------------------------------------------------
LEVELS = [(1, 10), (-1, 10), (1, 18), (1, 26), (-1, 33), (1, 34), (1, 60), (-1, 60), (1, 112), (-1, 112)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("base", [1.0, 1.375])
@pytest.mark.parametrize("sign,level", LEVELS)
@pytest.mark.parametrize("H,G,D,n,bs", [(2, 2, 64, 300, 16), (1, 4, 128, 20000, 32), (2, 12, 128, 700, 16), (1, 3, 256, 5000, 64)])
def test_logits_of_any_size(kvc, dt, base, sign, level, H, G, D, n, bs):
    """Keys of equal components and powers of two make the logits exact.  The largest one belongs to a third of the
    slots and the others lie so far below that their weight is 0: the output is the mean of the values there,
    however large the logits and whatever the scales of the pages."""
    B, half = 2, level // 2
    g = torch.Generator().manual_seed(1)
    best = torch.rand((B, H, n), generator=g) < 0.35
    best[..., 0] = True
    best = best.to(DEV)
    k = torch.where(best, 1.0, 0.5 if sign > 0 else 2.0)[..., None].expand(B, H, n, D) * base
    v = torch.randn((B, H, n, D), generator=g).to(torch.float8_e4m3fn).float().to(DEV)
    per = -(-n // bs)
    ks = torch.full((B, H, per), 2.0 ** (level - half), device=DEV)
    vs = torch.exp2(torch.randint(-9, 10, (B, H, per), generator=g).float()).to(DEV)
    c = Cache(kvc, k, v, ks, vs, bs)
    q = torch.full((B, H * G, D), sign * 2.0 ** half, dtype=dt, device=DEV)
    out, lse = decode(kvc, c, q, 1.0)
    w = best.double() / best.sum(dim=2, keepdim=True)
    mean, size = (torch.einsum("bhn,bhnd->bhd", w, x)[:, :, None].expand(B, H, G, D).reshape(B, H * G, D) for x in (c.v, c.v.abs()))
    # the sums, the exponential and the quotient, and the output's rounding; the weights are powers of two
    rel = (cut_sums(n, B * H) + 4) * 2.0 ** -23
    tol = rel * size + step(dt) * (mean.abs() + rel * size)
    assert bool(((out.double() - mean).abs() <= tol).all()), float(((out.double() - mean).abs() / tol).max())
    want = sign * base * 2.0 ** level * D + torch.log(best.sum(dim=2).double())[:, :, None].expand(B, H, G).reshape(B, H * G)
    # five roundings of the largest logit (its factor, its product, log2(e), the sum with the logarithm, ln(2)), the
    # logarithm of a sum of that many cut sums and its own two roundings
    assert bool(((lse.double() - want).abs() <= 2.0 ** -21 * want.abs() + rel + 2.0 ** -22 * math.log(n)).all())


@pytest.mark.parametrize("dt", TYPES)
def test_logits_among_the_lowest_numbers(kvc, dt):
    test_logits_of_any_size(kvc, dt, 1.25, -1, 121, 1, 4, 64, 300, 16)


# ------------------------------------------------------------------------------------------
def tails(kvc, dt, n, D, G, heavy, X, bs=32, sink_value=True):
    """The slots `heavy` have a logit X, the others 0; all values lie in [1, 2), those of the heavy slots are 0 in the
    first half of the dims, and everywhere without sink_value.  Returns the outputs' errors over their bounds.

    The logits are exact.  The weights' exponents take two roundings of at most X log2(e), their exponentials
    are 2^-22 off, each of two, and their own rounding is 2^-22 as two terms.  Both terms end at 2^-25, for a
    reference of 2^6 to 2^7: a light weight may be off by 2^-30 of a heavy one, or be lost, in the 16 steps of 16
    slots (32 with 64 dims) at most that share its reference."""
    k = torch.zeros((1, 1, n, D), device=DEV)
    k[:, :, heavy] = 1.0
    v = positive((1, 1, n, D), 3)
    v[:, :, heavy, : D // 2 if sink_value else D] = 0.0
    per = -(-n // bs)
    one = torch.ones((1, 1, per), device=DEV)
    c = Cache(kvc, k, v, one, one, bs)
    q = torch.ones((1, G, D), dtype=dt, device=DEV)
    scale = float(torch.tensor(X / D, dtype=torch.float32))
    out, lse = decode(kvc, c, q, scale)
    want, want_lse, _, size = attention(q[0].double(), c.k[0, 0], c.v[0, 0], scale)
    weight = X * 2.0 ** -22 + 2.0 ** -21 + 2.0 ** -22 + cut_sums(n, 1) * 2.0 ** -23
    light = math.exp(-float(want_lse[0]))
    small = len(heavy) * 16 * (32 if D == 64 else 16) * min(light, 2.0 ** -30 * light * math.exp(X)) * 2.0
    tol = weight * size + small + step(dt) * want.abs() * (1 + weight)
    assert bool(((lse[0].double() - want_lse).abs() <= weight + 2.0 ** -22 * want_lse.abs()).all())
    return float(((out[0].double() - want).abs() / tol).max())


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("X", [0.3, 3.0, 14.0, 21.83, 30.0, 40.0])
@pytest.mark.parametrize("D,G,heavy", [(64, 1, [0]), (128, 4, [0]), (128, 12, [70001]), (128, 2, [131071]), (256, 1, [5]),
                                       (64, 8, list(range(0, 131072, 1000)))])
def test_a_heavy_slot_and_a_hundred_thousand_light_ones(kvc, dt, X, D, G, heavy):
    """Weights of 2^-20 or 2^-31 of the largest, a hundred thousand times, are an output where the heavy slot's
    value is 0, and a part of it elsewhere.  With X = 0.3 all light weights are rounded alike."""
    assert tails(kvc, dt, 131072, D, G, heavy, X) <= 1.0


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("X", [50.0, 70.0])
def test_light_slots_alone(kvc, dt, X):
    """The heavy slot's value is 0 everywhere: the outputs are sums of weights of 2^-72 and 2^-101."""
    assert tails(kvc, dt, 20000, 128, 2, [0], X, sink_value=False) <= 1.0


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("D,G", [(64, 2), (128, 1), (128, 12), (256, 3)])
def test_logits_that_rise_and_fall(kvc, dt, D, G):
    """Logits of normal numbers times 12 and pages whose values differ by 2^24: the references move often."""
    B, H, n, bs = 3, 1, 3000, 16
    g = torch.Generator(device=DEV).manual_seed(4)
    k, v = (torch.randn((B, H, n, D), generator=g, device=DEV).to(torch.float8_e4m3fn).float() for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(-r, r + 1, (B, H, -(-n // bs)), generator=g, device=DEV).float()) for r in (1, 12))
    c = Cache(kvc, k, v, ks, vs, bs)
    q = (torch.randn((B, G, D), generator=g, device=DEV) * 12).to(dt)
    scale = 1.0 / math.sqrt(D)
    out, lse = decode(kvc, c, q, scale)
    for b in range(B):
        want, want_lse, x, size = attention(q[b].double(), c.k[b, 0], c.v[b, 0], scale)
        # a logit takes D products in sums that are cut (2^-23 each), and fp32 queries are 22 bits of the largest
        dx = scale * (D + 8) * 2.0 ** -23 * (q[b].double().abs() @ c.k[b, 0].abs().T) + x.abs() * 2.0 ** -22
        if dt == torch.float32:
            dx = dx + scale * 2.0 ** -22 * q[b].double().abs().amax(dim=1, keepdim=True) * c.k[b, 0].abs().sum(dim=1)
        weight = (torch.softmax(x, dim=1) * (2 * dx.amax(dim=1, keepdim=True) + dx)).sum(dim=1, keepdim=True)
        rel = weight + (x.amax() - x.amin()) * 2.0 ** -22 + 2.0 ** -20 + cut_sums(n, 1) * 2.0 ** -23
        tol = rel * size + step(dt) * want.abs() * (1 + rel)
        assert bool(((out[b].double() - want).abs() <= tol).all()), float(((out[b].double() - want).abs() / tol).max())
        assert bool(((lse[b].double() - want_lse).abs() <= rel[:, 0] + 2.0 ** -22 * want_lse.abs()).all())


@pytest.mark.parametrize("dt,D,G", [(torch.float32, 128, 2), (torch.bfloat16, 64, 8)])
def test_warps_of_a_thousand_steps(kvc, dt, D, G):
    """Thousands of sequences that list the same pages: a warp walks a whole row, whose sums of one sign
    are cut a thousand times or two."""
    n, bs, B = 16000, 32, 2560
    g = torch.Generator(device=DEV).manual_seed(5)
    k = torch.randn((1, 1, n, D), generator=g, device=DEV).to(torch.float8_e4m3fn).float()
    per = n // bs
    c = Cache(kvc, k, positive((1, 1, n, D), 6), *(torch.full((1, 1, per), 0.25, device=DEV) for _ in range(2)), bs)
    table, lens = c.table.expand(B, per).contiguous(), c.len.expand(B).contiguous()
    pt = kvc.page_table_view(table, c.nb.expand(B).contiguous(), lens, torch.zeros((B, per), device=DEV))
    few = torch.randn((8, G, D), generator=g, device=DEV).to(dt)
    q = few.repeat(B // 8, 1, 1)
    scale = 1.0 / math.sqrt(D)
    out = kvc.kvc_decode_attn_paged_q8(q, c.pool, pt, scale=scale)
    assert kvc.kvc_device_status() == 0
    for i in range(8):
        want, _, x, size = attention(few[i].double(), c.k[0, 0], c.v[0, 0], scale)
        dx = scale * (D + 8) * 2.0 ** -23 * (few[i].double().abs() @ c.k[0, 0].abs().T) + x.abs() * 2.0 ** -22
        if dt == torch.float32:
            dx = dx + scale * 2.0 ** -22 * few[i].double().abs().amax(dim=1, keepdim=True) * c.k[0, 0].abs().sum(dim=1)
        rel = (torch.softmax(x, dim=1) * (2 * dx.amax(dim=1, keepdim=True) + dx)).sum(dim=1, keepdim=True)
        rel = rel + 2.0 ** -20 + cut_sums(n, B) * 2.0 ** -23
        tol = rel * size + step(dt) * want.abs() * (1 + rel)
        err = (out[i::8].double() - want).abs()
        assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("D,G", [(64, 1), (128, 3), (128, 12), (256, 2)])
@pytest.mark.parametrize("X", [0.3, 1.9, 4.4])
def test_sums_that_cancel(kvc, dt, D, G, X):
    """One heavy slot whose value is the negative of what the others add up to: what is left shows the weights' own
    rounding, as two terms, whatever the queries' and outputs' type."""
    n, bs = 1008, 16
    k, v = torch.zeros((1, 1, n, D), device=DEV), torch.ones((1, 1, n, D), device=DEV)
    k[:, :, 0], v[:, :, 0], v[:, :, 1:bs] = 1.0, -1.0, 0.0
    one = torch.ones((1, 1, n // bs), device=DEV)
    vs = one.clone()
    vs[..., 0] = (n - bs) * math.exp(-X)
    c = Cache(kvc, k, v, one, vs, bs)
    scale = float(torch.tensor(X / D, dtype=torch.float32))
    out, _ = decode(kvc, c, torch.ones((1, G, D), dtype=dt, device=DEV), scale)
    want, _, _, size = attention(torch.ones((G, D), dtype=torch.float64, device=DEV), c.k[0, 0], c.v[0, 0], scale)
    assert bool((want.abs() <= 2.0 ** -20 * size).all())
    # as in tails(), where every product of 16 slots has weights of one size or two
    tol = (X * 2.0 ** -22 + 2.0 ** -21 + 2.0 ** -22 + cut_sums(n, 1) * 2.0 ** -23) * size
    assert bool(((out[0].double() - want).abs() <= tol * (1 + step(dt))).all()), float(((out[0].double() - want).abs() / tol).max())
