"""Refusals of the draft-tree and latent entry points, in the library and in the binding.  No GPU
needed: nothing here launches a kernel."""
import ctypes

import pytest
import torch

B_ = ctypes.byref


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_kvc_gb300 import build, kvc as k
    build.build()
    k.load()
    return k


def cache(kvc, **kw):
    c = kvc.kvc_cache()
    c.k = c.v = 4096
    c.dtype, c.batch, c.n_heads_kv, c.cap, c.d_head = kvc.KVC_BF16, 2, 2, 16, 128
    c.stride_b, c.stride_h, c.stride_slot = 2 * 16 * 128, 16 * 128, 128
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def latent(kvc, **kw):
    c = kvc.kvc_latent_cache()
    c.c, c.dtype, c.batch, c.cap, c.d_latent, c.d_rope = 4096, kvc.KVC_BF16, 2, 16, 512, 64
    c.stride_b, c.stride_slot = 16 * 576, 576
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def draft(kvc, **kw):
    d = kvc.kvc_draft()
    d.k = d.v = 4096
    d.n_draft = 4
    for k, v in kw.items():
        setattr(d, k, v)
    return d


OK, ARG, SHAPE, ALIGN, CAP, WS = 0, 1, 2, 3, 4, 6


@pytest.mark.parametrize("want,cache_kw,draft_kw,call", [
    (ARG, {"k": None}, {}, {}), (SHAPE, {"d_head": 96}, {}, {}), (ALIGN, {"k": 4104}, {}, {}),
    (SHAPE, {"stride_slot": 64}, {}, {}), (ALIGN, {"stride_slot": 132}, {}, {}),
    (SHAPE, {}, {"n_draft": 0}, {}), (SHAPE, {}, {"n_draft": 65}, {}), (ARG, {}, {"v": None}, {}),
    (ARG, {}, {"k": None}, {}), (ALIGN, {}, {"k": 4100}, {}), (ALIGN, {}, {"mask": 4100}, {}),
    (ALIGN, {}, {"count": 4098}, {}), (SHAPE, {}, {}, {"hq": 3}), (SHAPE, {}, {}, {"hq": 0}),
    (SHAPE, {}, {}, {"hq": 130}), (ARG, {}, {}, {"q": None}), (ARG, {}, {}, {"out": None}),
    (ALIGN, {}, {}, {"q": 4104}), (ALIGN, {}, {}, {"out": 4104}), (ALIGN, {}, {}, {"lse": 4098}),
    (ARG, {}, {}, {"scale": float("nan")}), (CAP, {}, {}, {"n_valid": 17}), (CAP, {}, {}, {"n_valid": -1}),
])
def test_tree_refusals(kvc, want, cache_kw, draft_kw, call):
    a = dict(q=4096, hq=4, len=None, n_valid=4, scale=1.0, out=4096, lse=None)
    a.update(call)
    st = kvc.load().kvc_decode_attn_tree(a["q"], a["hq"], B_(cache(kvc, **cache_kw)), a["len"], a["n_valid"],
                                         B_(draft(kvc, **draft_kw)), a["scale"], a["out"], a["lse"], None, 0,
                                         None)
    assert st == want and kvc.kvc_last_error()


@pytest.mark.parametrize("want,cache_kw,draft_kw,call", [
    (ARG, {"c": None}, {}, {}), (ARG, {"dtype": 5}, {}, {}), (SHAPE, {"d_latent": 384}, {}, {}),
    (SHAPE, {"d_rope": 12}, {}, {}), (SHAPE, {"d_rope": 72}, {}, {}), (SHAPE, {"stride_slot": 568}, {}, {}),
    (ALIGN, {"stride_slot": 580}, {}, {}), (ALIGN, {"c": 4104}, {}, {}), (SHAPE, {"batch": 0}, {}, {}),
    (SHAPE, {}, {"n_draft": 65}, {}), (SHAPE, {}, {}, {"hq": 257}), (SHAPE, {}, {}, {"hq": 0}),
    (CAP, {}, {}, {"n_valid": 17}), (ARG, {}, {}, {"q": None}),
])
def test_latent_refusals(kvc, want, cache_kw, draft_kw, call):
    a = dict(q=4096, hq=16, n_valid=4)
    a.update(call)
    st = kvc.load().kvc_decode_attn_latent(a["q"], a["hq"], B_(latent(kvc, **cache_kw)), None, a["n_valid"],
                                           B_(draft(kvc, **draft_kw)), 1.0, 4096, None, None, 0, None)
    assert st == want and kvc.kvc_last_error()


def test_more_tiles_than_a_block_counts_is_refused(kvc):
    """Broadcast sequences (stride 0) of the largest capacity, for tree and latent attention."""
    big = {"batch": 1 << 21, "cap": 2 ** 31 - 1, "stride_b": 0, "stride_slot": 576}
    st = kvc.load().kvc_decode_attn_latent(4096, 16, B_(latent(kvc, **big)), None, 4, B_(draft(kvc)), 1.0,
                                           4096, None, None, 0, None)
    assert st == SHAPE and "too large" in kvc.kvc_last_error()
    big = {"batch": 1 << 21, "cap": 2 ** 31 - 1, "stride_b": 0, "stride_h": 0}
    st = kvc.load().kvc_decode_attn_tree(4096, 4, B_(cache(kvc, **big)), None, 4, B_(draft(kvc)), 1.0,
                                         4096, None, None, 0, None)
    assert st == SHAPE and "too large" in kvc.kvc_last_error()


def test_accept_refusals_before_launch(kvc):
    lib = kvc.load()
    c, d, lt = cache(kvc), draft(kvc), latent(kvc)
    assert lib.kvc_tree_accept(B_(c), 4096, B_(d), None, 4096, None) == ARG
    assert lib.kvc_tree_accept(B_(c), None, B_(d), 4096, 4096, None) == ARG
    assert lib.kvc_tree_accept(B_(c), 4096, B_(d), 4096, None, None) == ARG
    assert lib.kvc_tree_accept(B_(c), 4096, B_(draft(kvc, k=None, v=None)), 4096, 4096, None) == ARG
    assert lib.kvc_tree_accept(B_(c), 4096, None, 4096, 4096, None) == ARG
    assert lib.kvc_latent_accept(B_(lt), 4096, B_(draft(kvc, k=None)), 4096, 4096, None) == ARG
    assert lib.kvc_latent_accept(B_(latent(kvc, d_latent=500)), 4096, B_(d), 4096, 4096, None) == SHAPE
    pool, pt, fp = kvc.kvc_block_pool(), kvc.kvc_page_table(), kvc.kvc_free_pool()
    pool.k = pool.v = 4096
    pool.dtype, pool.n_blocks, pool.n_heads_kv, pool.block_size, pool.d_head = kvc.KVC_BF16, 8, 2, 16, 128
    pt.table = pt.n_blocks = pt.len = pt.score = 4096
    pt.batch, pt.max_blocks = 2, 4
    fp.ids, fp.top, fp.capacity = 4096, 4096, 8
    assert lib.kvc_tree_accept_paged(B_(pool), B_(pt), B_(fp), B_(d), 4096, 4096, None, None) == ARG
    fp.capacity = 0
    assert lib.kvc_tree_accept_paged(B_(pool), B_(pt), B_(fp), B_(d), 4096, 4096, 4096, None) == ARG
    fp.capacity, pool.d_head = 8, 80
    assert lib.kvc_tree_accept_paged(B_(pool), B_(pt), B_(fp), B_(d), 4096, 4096, 4096, None) == SHAPE
    assert lib.kvc_decode_attn_tree_paged(4096, 4, B_(pool), B_(pt), B_(d), 1.0, 4096, None, None, 0, None) == SHAPE
    pool.d_head, pool.block_size = 128, 0
    assert lib.kvc_decode_attn_tree_paged(4096, 4, B_(pool), B_(pt), B_(d), 1.0, 4096, None, None, 0, None) == SHAPE


def test_expand_refusals(kvc):
    lib = kvc.load()
    lt, dst = latent(kvc), cache(kvc)

    def call(lat=lt, d=dst, n=4, wk=4096, wv=4096):
        return lib.kvc_latent_expand(B_(lat), None, n, wk, wv, B_(d), None)

    assert call(n=17) == CAP and call(n=-1) == CAP
    assert call(d=cache(kvc, cap=3)) == CAP
    assert call(wk=None) == ARG and call(wv=4104) == ALIGN
    assert call(d=cache(kvc, batch=3)) == SHAPE and call(d=cache(kvc, dtype=kvc.KVC_F32)) == SHAPE
    assert call(d=cache(kvc, d_head=64, stride_slot=64)) == SHAPE          # d_rope 64 leaves no key
    assert call(d=cache(kvc, n_heads_kv=40000)) == SHAPE
    assert call(lat=latent(kvc, d_rope=4)) == SHAPE


def test_workspace_queries(kvc):
    lib = kvc.load()
    tree, lat = lib.kvc_decode_attn_tree_workspace_bytes, lib.kvc_decode_attn_latent_workspace_bytes
    assert tree(1, 32, 8, 128, 16, kvc.KVC_BF16) > 0 and tree(1, 32, 8, 128, 16, kvc.KVC_F32) > 0
    assert lat(1, 128, 512, 64, 4, kvc.KVC_BF16) > 0
    for bad in ((0, 32, 8, 128, 4, 1), (1, 30, 8, 128, 4, 1), (1, 32, 8, 100, 4, 1), (1, 32, 8, 128, 0, 1),
                (1, 32, 8, 128, 65, 1), (1, 32, 8, 128, 4, 2), (1, 520, 8, 128, 4, 1), (1, 0, 8, 128, 4, 1)):
        assert tree(*bad) == 0
    for bad in ((0, 16, 512, 64, 1, 1), (1, 257, 512, 64, 1, 1), (1, 16, 500, 64, 1, 1), (1, 16, 512, 4, 1, 1),
                (1, 16, 512, 64, 65, 1), (1, 16, 512, 64, 1, 3)):
        assert lat(*bad) == 0


def test_binding_checks_its_tensors(kvc):
    k = torch.zeros(2, 4, 2, 64)
    with pytest.raises(ValueError):
        kvc.make_draft(k)                                      # keys without values
    with pytest.raises(ValueError):
        kvc.make_draft(k, k.transpose(0, 1))
    with pytest.raises(ValueError):
        kvc.make_draft(k, k, mask=torch.zeros(2, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        kvc.make_draft(k, k, count=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        kvc.make_draft(k, k, n_draft=5)
    with pytest.raises(ValueError):
        kvc.make_draft(mask=torch.zeros(2, 4, dtype=torch.int64), n_draft=4)
    with pytest.raises(ValueError):
        kvc.make_draft()
    d = kvc.make_draft(k, k)
    assert d.n_draft == 4
    c = kvc.cache_view(torch.zeros(2, 2, 9, 64), torch.zeros(2, 2, 9, 64))
    q = torch.zeros(2, 4, 4, 64)
    for bad in (q[:, :3], q.double(), q[..., :32].contiguous(), q.transpose(1, 2), torch.zeros(3, 4, 4, 64)):
        with pytest.raises(ValueError):
            kvc.kvc_decode_attn_tree(bad, c, d, scale=1.0, n_valid=3)
    with pytest.raises(ValueError):
        kvc.kvc_decode_attn_tree(q, c, d, scale=1.0, len=torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError):
        kvc.kvc_decode_attn_tree(q, c, d, scale=1.0, n_valid=3, out=torch.zeros(2, 4, 4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        kvc.kvc_decode_attn_tree(q, c, d, scale=1.0, n_valid=3, lse=torch.zeros(2, 4))
    with pytest.raises(ValueError):                            # drafted rows of another head count
        kvc.kvc_decode_attn_tree(q, kvc.cache_view(*[torch.zeros(2, 4, 9, 64)] * 2), d, scale=1.0, n_valid=3)
    with pytest.raises(ValueError):
        kvc.latent_cache_view(torch.zeros(2, 5, 192)[..., ::2], 64)
    with pytest.raises(ValueError):
        kvc.latent_cache_view(torch.zeros(2, 5, 192), 200)
    lat = kvc.latent_cache_view(torch.zeros(2, 5, 192), 128)
    with pytest.raises(ValueError):
        kvc.kvc_decode_attn_latent(torch.zeros(2, 4, 8, 192), lat, d, scale=1.0, n_valid=3)
    with pytest.raises(ValueError):
        kvc.kvc_tree_accept(c, torch.zeros(2, 2, dtype=torch.int32), d, torch.zeros(2, 3, dtype=torch.int32),
                            torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        kvc.kvc_tree_accept(c, torch.zeros(2, 2, dtype=torch.int64), d, torch.zeros(2, 4, dtype=torch.int32),
                            torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        kvc.kvc_latent_expand(lat, torch.zeros(2, 1, 128), torch.zeros(2, 64, 128), c, n_valid=3)


def test_descriptors_of_another_device_are_refused(kvc, monkeypatch):
    """Any tensor that a descriptor keeps: the first or a later one, in a tuple or alone."""
    class On:
        def __init__(self, index):
            self.device = f"cuda:{index}"
            self.get_device = lambda: index

    class View:
        pass

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    v = View()
    kvc._on_current(0, v, "q")                              # made without tensors: nothing known
    for kept in ((On(0), On(0)), (On(0), None), On(0)):
        v._keep = kept
        kvc._on_current(0, v, "q")
    for kept in ((On(0), On(1)), (On(1), None), On(1), (On(0), On(0), On(0), On(-1))):
        v._keep = kept
        with pytest.raises(ValueError, match="View"):
            kvc._on_current(0, v, "q")
    with pytest.raises(ValueError, match="current"):
        kvc._on_current(1, View(), "q")
    with pytest.raises(ValueError, match="CPU"):
        kvc._on_current(-1, View(), "q")
