"""Norms and rotation of queries and keys against the formula in 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_kvc_gb300 import kvc as k
    k.load()
    return k


def rows(seed, dt, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dt)


def reference(x, w, eps, cs, pos):
    """(result, the size that its fp32 errors are relative to)"""
    y = x.double()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(dim=-1, keepdim=True) + eps) * w.double()
    size = y.abs()
    if cs is not None:
        h = cs.shape[2]
        c, s = cs.double()[pos.long()][:, None].unbind(dim=2)
        a, b = y[..., :h], y[..., h:2 * h]
        m = a.abs() + b.abs()
        y = torch.cat([a * c - b * s, b * c + a * s, y[..., 2 * h:]], dim=-1)
        size = torch.cat([m, m, size[..., 2 * h:]], dim=-1)
    return y, size


def check(got, x, w, eps, cs, pos):
    want, size = reference(x, w, eps, cs, pos)
    # half a step of the type, and fp32: the sum of squares (at most 8 + 5 roundings of 2^-24, halved by
    # the root), the root's 2 ulp, two products, two more and a sum of the rotation: under 24 * 2^-24
    tol = torch.finfo(x.dtype).eps / 2 * want.abs() + 24 * 2.0 ** -24 * size + 1e-30
    assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [
    (1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (3, 5, 3, 256, 256), (17, 24, 4, 256, 64), (130, 6, 1, 64, 16),
    (7, 33, 17, 128, 96), (257, 2, 2, 128, 32), (5, 7, 2, 64, 48), (64, 9, 9, 256, 144), (2, 40, 40, 64, 0)])
def test_against_the_formula(kvc, dt, T, Hq, Hkv, D, rot):
    q, k = rows(1, dt, T, Hq, D) * 3, rows(2, dt, T, Hkv, D)
    wq, wk = rows(3, dt, D), rows(4, dt, D)
    cs = kvc.kvc_rope_table(300, rot).to(DEV) if rot else None
    pos = torch.randint(0, 300, (T,), device=DEV, dtype=torch.int32) if rot else None
    a, b = kvc.kvc_qk_norm_rope(q, k, w_q=wq, w_k=wk, eps=1e-5, cos_sin=cs, pos=pos)
    check(a, q, wq, 1e-5, cs, pos)
    check(b, k, wk, 1e-5, cs, pos)
    assert kvc.kvc_device_status() == 0


def test_one_weight_or_none(kvc):
    q, k = rows(5, torch.bfloat16, 9, 4, 128), rows(6, torch.bfloat16, 9, 2, 128)
    cs, pos = kvc.kvc_rope_table(9, 128).to(DEV), torch.arange(9, device=DEV, dtype=torch.int32)
    w = rows(7, torch.bfloat16, 128)
    for wq, wk in ((w, None), (None, w), (None, None)):
        a, b = kvc.kvc_qk_norm_rope(q, k, w_q=wq, w_k=wk, cos_sin=cs, pos=pos)
        check(a, q, wq, 1e-6, cs, pos)
        check(b, k, wk, 1e-6, cs, pos)


def test_rotation_keeps_distances_and_leaves_the_rest(kvc):
    """Position 0 rotates by nothing; rows behind d_rot are only normed."""
    q, k = rows(8, torch.float32, 6, 2, 128), rows(9, torch.float32, 6, 2, 128)
    cs = kvc.kvc_rope_table(50, 64).to(DEV)
    zero = torch.zeros(6, device=DEV, dtype=torch.int32)
    a, b = kvc.kvc_qk_norm_rope(q, k, cos_sin=cs, pos=zero)
    assert torch.equal(a, q) and torch.equal(b, k)
    a, _ = kvc.kvc_qk_norm_rope(q, k, cos_sin=cs, pos=zero + 49)
    assert torch.equal(a[..., 64:], q[..., 64:]) and not torch.equal(a[..., :64], q[..., :64])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_strided_rows_and_in_place(kvc, dt):
    """Queries, keys and values in one projection's output; outputs in place and transposed."""
    T, Hq, Hkv, D = 37, 6, 2, 64
    qkv = rows(10, dt, T, Hq + 2 * Hkv, D)
    before = qkv.clone()
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    w = rows(11, dt, D)
    cs, pos = kvc.kvc_rope_table(64, 32).to(DEV), torch.arange(T, device=DEV, dtype=torch.int32)
    fresh = kvc.kvc_qk_norm_rope(q, k, w_q=w, w_k=w, cos_sin=cs, pos=pos)
    assert torch.equal(qkv, before)
    turned = torch.zeros((Hq, T, D), device=DEV, dtype=dt).transpose(0, 1)
    kvc.kvc_qk_norm_rope(q, k, w_q=w, w_k=w, cos_sin=cs, pos=pos, q_out=turned)
    assert torch.equal(turned, fresh[0])
    kvc.kvc_qk_norm_rope(q, k, w_q=w, w_k=w, cos_sin=cs, pos=pos, q_out=q, k_out=k)
    assert torch.equal(q, fresh[0]) and torch.equal(k, fresh[1])
    assert torch.equal(qkv[:, Hq + Hkv:], before[:, Hq + Hkv:])


def test_bad_position_leaves_the_token(kvc):
    q, k = rows(12, torch.bfloat16, 4, 3, 64), rows(13, torch.bfloat16, 4, 1, 64)
    cs = kvc.kvc_rope_table(10, 64).to(DEV)
    pos = torch.tensor([3, -1, 10, 9], device=DEV, dtype=torch.int32)
    a, b = (torch.full_like(x, 7) for x in (q, k))
    kvc.kvc_qk_norm_rope(q, k, cos_sin=cs, pos=pos, q_out=a, k_out=b)
    assert kvc.kvc_device_status() == 4
    assert bool((a[1:3] == 7).all()) and bool((b[1:3] == 7).all())
    keep = torch.tensor([0, 3], device=DEV)
    check(a[keep], q[keep], None, 0, cs, pos[keep])
    check(b[keep], k[keep], None, 0, cs, pos[keep])


def test_no_tokens_zeros_and_non_finite(kvc):
    w = rows(14, torch.float32, 64)
    e = torch.empty((0, 4, 64), device=DEV)
    a, b = kvc.kvc_qk_norm_rope(e, e, w_q=w, w_k=w)
    assert a.shape == b.shape == (0, 4, 64)
    q = rows(15, torch.float32, 5, 2, 64)
    q[1, 0] = 0
    q[2, 1, 5] = float("nan")
    a, _ = kvc.kvc_qk_norm_rope(q, q.clone(), w_q=w, w_k=w)
    assert bool((a[1, 0] == 0).all()) and bool(a[2, 1].isnan().all())
    ok = torch.ones((5, 2), dtype=torch.bool, device=DEV)
    ok[2, 1] = False
    assert bool(a[ok].isfinite().all())


def test_captured_and_on_another_stream(kvc):
    q, k = rows(16, torch.bfloat16, 16, 8, 128), rows(17, torch.bfloat16, 16, 2, 128)
    w = rows(18, torch.bfloat16, 128)
    want = kvc.kvc_qk_norm_rope(q, k, w_q=w, w_k=w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = kvc.kvc_qk_norm_rope(q, k, w_q=w, w_k=w, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a, b = torch.zeros_like(q), torch.zeros_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.kvc_qk_norm_rope(q, k, w_q=w, w_k=w, q_out=a, k_out=b)
    for i in range(3):
        q.copy_(rows(20 + i, torch.bfloat16, 16, 8, 128))
        graph.replay()
        assert torch.equal(a, kvc.kvc_qk_norm_rope(q, k, w_q=w, w_k=w)[0])


def test_many_tokens(kvc):
    """More rows than a grid of one wave; offsets beyond 2^31 bytes."""
    T, Hq, Hkv, D = 70001, 32, 8, 128
    q, k = rows(30, torch.bfloat16, T, Hq, D), rows(31, torch.bfloat16, T, Hkv, D)
    w = rows(32, torch.bfloat16, D)
    cs = kvc.kvc_rope_table(4096, D).to(DEV)
    pos = (torch.arange(T, device=DEV) % 4096).to(torch.int32)
    a, b = kvc.kvc_qk_norm_rope(q, k, w_q=w, w_k=w, cos_sin=cs, pos=pos)
    for at in (slice(0, 9), slice(34990, 35011), slice(T - 9, T)):
        check(a[at], q[at], w, 1e-6, cs, pos[at])
        check(b[at], k[at], w, 1e-6, cs, pos[at])


@pytest.mark.parametrize("dt,T,Hq,Hkv,D,rot", [
    (torch.bfloat16, 15001, 8, 1, 64, 64), (torch.bfloat16, 20003, 3, 1, 128, 64), (torch.bfloat16, 8001, 32, 8, 128, 128),
    (torch.float32, 15005, 4, 1, 64, 16), (torch.float32, 3649, 5, 3, 128, 0), (torch.bfloat16, 3649, 4, 4, 256, 256),
    (torch.bfloat16, 14591, 1, 1, 64, 64)])
def test_every_row_of_long_prompts(kvc, dt, T, Hq, Hkv, D, rot):
    """More tokens than warps: whole rounds of them, then the rest; few heads, whose tokens lie side by side."""
    q, k = rows(40, dt, T, Hq, D), rows(41, dt, T, Hkv, D)
    wq, wk = rows(42, dt, D), rows(43, dt, D)
    cs = kvc.kvc_rope_table(500, rot).to(DEV) if rot else None
    pos = torch.randint(0, 500, (T,), device=DEV, dtype=torch.int32) if rot else None
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    if rot:
        bad[[0, 5, T // 2, T - 1]] = True
        pos[bad] = 500
    a, b = torch.full_like(q, 7), torch.full_like(k, 7)
    kvc.kvc_qk_norm_rope(q, k, w_q=wq, w_k=wk, cos_sin=cs, pos=pos, q_out=a, k_out=b)
    assert kvc.kvc_device_status() == (4 if rot else 0)
    assert bool((a[bad] == 7).all()) and bool((b[bad] == 7).all())
    ok = ~bad
    check(a[ok], q[ok], wq, 1e-6, cs, pos[ok] if rot else None)
    check(b[ok], k[ok], wk, 1e-6, cs, pos[ok] if rot else None)
