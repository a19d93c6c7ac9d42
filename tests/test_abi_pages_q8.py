"""Refusals of the norms with rotation, the 8-bit pages and the calls on pages, in the library and in the
binding.  No GPU needed: nothing here launches a kernel."""
import ctypes

import pytest
import torch

from test_abi_tree_arguments import Elsewhere, Lib, OnDevice

B_ = ctypes.byref
OK, ARG, SHAPE, ALIGN, CAP, WS = 0, 1, 2, 3, 4, 6
I32, F32, BF16, U8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8


@pytest.fixture(scope="module")
def lib():
    from kv_cache_compression_kvc_gb300 import build, kvc as k
    build.build()
    return k.load()


@pytest.fixture(scope="module")
def K():
    from kv_cache_compression_kvc_gb300 import kvc as k
    return k


# ------------------------------------------------------------------------------------------
# The library.


def rows(K, **kw):
    r = K.kvc_qk_rows()
    r.q = r.k = r.q_out = r.k_out = 4096
    r.dtype, r.n_tokens, r.n_heads_q, r.n_heads_kv, r.d_head, r.d_rot = K.KVC_BF16, 4, 8, 2, 128, 64
    r.q_stride_token = r.q_out_stride_token = 1024
    r.k_stride_token = r.k_out_stride_token = 256
    r.q_stride_head = r.q_out_stride_head = r.k_stride_head = r.k_out_stride_head = 128
    for k, v in kw.items():
        setattr(r, k, v)
    return r


@pytest.mark.parametrize("want,kw,call", [
    (ARG, {"q": None}, {}), (ARG, {"k": None}, {}), (ARG, {"q_out": None}, {}), (ARG, {"k_out": None}, {}),
    (ARG, {"dtype": 2}, {}), (SHAPE, {"n_tokens": -1}, {}), (SHAPE, {"n_heads_q": 0}, {}), (SHAPE, {"n_heads_kv": 0}, {}),
    (SHAPE, {"d_head": 96}, {}), (SHAPE, {"d_rot": 8}, {}), (SHAPE, {"d_rot": 24}, {}), (SHAPE, {"d_rot": 144}, {}),
    (ALIGN, {"q": 4104}, {}), (ALIGN, {"k_out": 4104}, {}), (ALIGN, {"q_stride_token": 1028}, {}),
    (ALIGN, {"k_stride_head": 132}, {}), (SHAPE, {"q_stride_head": 64}, {}), (SHAPE, {"q_stride_token": -1024}, {}),
    (SHAPE, {"q_out": 8192, "q_out_stride_token": 512}, {}), (SHAPE, {"q_out": 8192, "q_out_stride_head": 0}, {}),
    (SHAPE, {"k_out": 8192, "k_out_stride_token": 128, "k_out_stride_head": 128}, {}),
    (SHAPE, {"q_out_stride_token": 2048}, {}), (SHAPE, {"n_tokens": 2 ** 31 - 1, "q_out": 8192, "k_out": 8192}, {}),
    (ARG, {}, {"w_q": None, "w_k": None, "cos_sin": None}), (ARG, {}, {"pos": None}), (SHAPE, {}, {"n_pos": 0}),
    (ALIGN, {}, {"w_q": 4104}), (ALIGN, {}, {"w_k": 4104}), (ALIGN, {}, {"cos_sin": 4104}), (ALIGN, {}, {"pos": 4098}),
    (ARG, {}, {"eps": -1e-6}), (ARG, {}, {"eps": float("nan")}), (ARG, {}, {"eps": float("inf")}),
])
def test_norm_refusals(lib, K, want, kw, call):
    a = dict(w_q=4096, w_k=4096, eps=1e-6, cos_sin=4096, pos=4096, n_pos=16)
    a.update(call)
    st = lib.kvc_qk_norm_rope(B_(rows(K, **kw)), a["w_q"], a["w_k"], a["eps"], a["cos_sin"], a["pos"], a["n_pos"], None)
    assert st == want and lib.kvc_last_error()
    assert lib.kvc_qk_norm_rope(None, 4096, 4096, 1e-6, None, None, 0, None) == ARG


def test_norm_of_no_tokens_launches_nothing(lib, K):
    assert lib.kvc_qk_norm_rope(B_(rows(K, n_tokens=0, q=None, k=None)), 4096, 4096, 1e-6, 4096, 4096, 16, None) == OK


def pool8(K, **kw):
    p = K.kvc_block_pool_q8()
    p.pages.k = p.pages.v = p.k_scale = p.v_scale = 4096
    p.pages.dtype, p.pages.n_blocks, p.pages.n_heads_kv, p.pages.block_size, p.pages.d_head = K.KVC_E4M3, 8, 2, 16, 128
    for k, v in kw.items():
        setattr(p if k.endswith("scale") else p.pages, k, v)
    return p


def table(K, **kw):
    pt = K.kvc_page_table()
    pt.table = pt.n_blocks = pt.len = pt.score = 4096
    pt.batch, pt.max_blocks = 2, 4
    for k, v in kw.items():
        setattr(pt, k, v)
    return pt


def stack(K, **kw):
    fp = K.kvc_free_pool()
    fp.ids, fp.top, fp.capacity = 4096, 4096, 8
    for k, v in kw.items():
        setattr(fp, k, v)
    return fp


BAD_POOL = [(ARG, {"k": None}), (ARG, {"v": None}), (ARG, {"k_scale": None}), (ARG, {"v_scale": None}), (ARG, {"dtype": 1}),
            (ARG, {"dtype": 3}), (SHAPE, {"n_blocks": 0}), (SHAPE, {"n_heads_kv": 0}), (SHAPE, {"block_size": 0}),
            (SHAPE, {"block_size": 24}), (SHAPE, {"block_size": 1040}), (SHAPE, {"d_head": 96}), (ALIGN, {"k": 4104}),
            (ALIGN, {"k_scale": 4098})]
BAD_TABLE = [(ARG, {"table": None}), (ARG, {"n_blocks": None}), (ARG, {"len": None}), (ARG, {"score": None}),
             (SHAPE, {"batch": 0}), (SHAPE, {"max_blocks": 0}), (SHAPE, {"max_blocks": 2 ** 30})]
BAD_STACK = [(ARG, {"ids": None}), (ARG, {"top": None}), (ARG, {"capacity": 0})]


def cases(own, tables=True, stacks=True):
    out = [(w, {"pool": kw}) for w, kw in BAD_POOL]
    out += [(w, {"table": kw}) for w, kw in BAD_TABLE] if tables else []
    out += [(w, {"stack": kw}) for w, kw in BAD_STACK] if stacks else []
    return out + own


@pytest.mark.parametrize("want,kw", cases([
    (ARG, {"k": None}), (ARG, {"v": None}), (ALIGN, {"k": 4104}), (ARG, {"dtype": 2}), (SHAPE, {"n": -1}),
    (SHAPE, {"n": 3, "cu": None}), (SHAPE, {"head": 64}), (ALIGN, {"token": 260}), (ALIGN, {"cu": 4098}),
    (ALIGN, {"appended": 4098}), (WS, {"ws": None}), (WS, {"wb": 255}), (WS, {"ws": 4096 + 128}),
    (SHAPE, {"n": 2 ** 31 - 1, "wb": 2 ** 40, "pool": {"n_heads_kv": 2 ** 10}})]))
def test_append_refusals(lib, K, want, kw):
    a = dict(k=4096, v=4096, dtype=K.KVC_BF16, n=5, token=256, head=128, cu=4096, appended=None, ws=4096, wb=1 << 20)
    a.update({k: v for k, v in kw.items() if k not in ("pool", "table", "stack")})
    st = lib.kvc_paged_append_q8(B_(pool8(K, **kw.get("pool", {}))), B_(table(K, **kw.get("table", {}))),
                                 B_(stack(K, **kw.get("stack", {}))), a["k"], a["v"], a["dtype"], a["n"], a["token"],
                                 a["head"], a["cu"], a["appended"], a["ws"], a["wb"], None)
    assert st == want and lib.kvc_last_error()


@pytest.mark.parametrize("want,kw", cases([
    (ARG, {"q": None}), (ARG, {"out": None}), (ARG, {"dtype": 2}), (ALIGN, {"q": 4104}), (ALIGN, {"out": 4104}),
    (ALIGN, {"lse": 4098}), (ALIGN, {"logits": 4098}), (CAP, {"logits": 4096, "stride": 63}), (SHAPE, {"hq": 3}),
    (SHAPE, {"hq": 0}), (SHAPE, {"hq": -2}), (ARG, {"scale": float("inf")}), (ARG, {"scale": float("nan")}),
    (WS, {"ws": None}), (WS, {"ws": 4096 + 16})], stacks=False))
def test_decode_refusals(lib, K, want, kw):
    a = dict(q=4096, dtype=K.KVC_BF16, hq=8, scale=1.0, out=4096, logits=None, stride=0, lse=None, ws=4096, wb=1 << 30)
    a.update({k: v for k, v in kw.items() if k not in ("pool", "table")})
    st = lib.kvc_decode_attn_paged_q8(a["q"], a["dtype"], a["hq"], B_(pool8(K, **kw.get("pool", {}))),
                                      B_(table(K, **kw.get("table", {}))), a["scale"], a["out"], a["logits"], a["stride"],
                                      a["lse"], a["ws"], a["wb"], None)
    assert st == want and lib.kvc_last_error()


@pytest.mark.parametrize("which", ["reorder", "compact"])
@pytest.mark.parametrize("want,kw", cases([
    (WS, {"ws": None}), (WS, {"wb": 128}), (WS, {"ws": 4096 + 16}), (ALIGN, {"shares": 4098}), (ALIGN, {"pos": 4098}),
    (ARG, {"last": None}), (ALIGN, {"last": 4097}), (ARG, {"plain": True, "ks": 4096}), (ARG, {"plain": True, "vs": 4096})]))
def test_page_refusals(lib, K, which, want, kw):
    p = pool8(K, **kw.get("pool", {}))
    a = dict(ks=p.k_scale, vs=p.v_scale, shares=4096, pos=None, last=4096, ws=4096, wb=1 << 20)
    if kw.get("plain"):
        p.pages.dtype, a["ks"], a["vs"] = K.KVC_BF16, None, None
    elif p.pages.dtype == 1:
        a["ks"] = 4096                           # bf16 pages with scales
    a.update({k: v for k, v in kw.items() if k not in ("pool", "table", "stack", "plain")})
    fn = lib.kvc_pages_reorder if which == "reorder" else lib.kvc_pages_compact
    st = fn(B_(p.pages), a["ks"], a["vs"], B_(table(K, **kw.get("table", {}))), B_(stack(K, **kw.get("stack", {}))),
            a["shares"], a["pos"], a["last"], a["ws"], a["wb"], None)
    assert st == want and lib.kvc_last_error()


def test_page_limits(lib, K):
    p = pool8(K)
    args = (p.k_scale, p.v_scale)
    assert lib.kvc_pages_reorder(B_(p.pages), *args, B_(table(K)), B_(stack(K)), None, None, 4096, 4096, 1 << 20, None) == ARG
    assert lib.kvc_pages_reorder(B_(p.pages), *args, B_(table(K, batch=8193)), B_(stack(K)), 4096, None, 4096, 4096,
                                 1 << 30, None) == SHAPE
    assert lib.kvc_pages_compact(B_(pool8(K, n_blocks=(1 << 20) + 1).pages), *args, B_(table(K)), B_(stack(K)), None, None,
                                 4096, 4096, 1 << 30, None) == SHAPE


def test_other_paged_calls_refuse_8_bit_pages(lib, K):
    pages, pt = pool8(K).pages, table(K)
    d = K.kvc_draft()
    d.n_draft = 1
    assert lib.kvc_paged_append(B_(pages), B_(pt), B_(stack(K)), 4096, 4096, None, None, None) == ARG
    assert lib.kvc_decode_attn_paged(4096, 2, B_(pages), B_(pt), 1.0, 4096, None, 0, None, 4096, 1 << 20, 0, None) == ARG
    assert lib.kvc_decode_attn_tree_paged(4096, 2, B_(pages), B_(pt), B_(d), 1.0, 4096, None, 4096, 1 << 20, None) == ARG


def test_workspace_queries(lib, K):
    app, dec, pag = (lib.kvc_paged_append_q8_workspace_bytes, lib.kvc_decode_attn_paged_q8_workspace_bytes,
                     lib.kvc_pages_workspace_bytes)
    assert app(4, 0, 16) >= 256 and app(4, 100, 16) >= 256 + 14 * 16 and pag(4, 8, 100) > 0
    assert dec(1, 8, 2, 64, K.KVC_BF16) > 0 and dec(2, 8, 2, 256, K.KVC_F32) > 0
    for bad in ((0, 4, 16), (1, -1, 16), (1, 4, 0)):
        assert app(*bad) == 0
    for bad in ((0, 8, 2, 64, 1), (1, 7, 2, 64, 1), (1, 0, 2, 64, 1), (1, 8, 0, 64, 1), (1, 8, 2, 0, 1)):
        assert dec(*bad) == 0
    for bad in ((0, 8, 8), (1, 0, 8), (1, 8, 0)):
        assert pag(*bad) == 0


# ------------------------------------------------------------------------------------------
# The binding.

B, HQ, H, D, BS, NB, MB, T = 2, 4, 2, 64, 16, 9, 3, 5


@pytest.fixture
def kvc(monkeypatch):
    from kv_cache_compression_kvc_gb300 import kvc as k
    stub = Lib()
    monkeypatch.setattr(k, "_lib", stub)
    monkeypatch.setattr(k, "load", lambda: stub)
    monkeypatch.setattr(k, "_on_current", k._beside)
    monkeypatch.setattr(k, "_raw_stream", lambda *a: 0)
    k.stub_calls = stub.calls
    yield k
    del k.stub_calls


def q8(k, **kw):
    a = dict(k_pool=torch.zeros(H, NB, BS, D, dtype=U8), v_pool=torch.zeros(H, NB, BS, D, dtype=U8),
             k_scale=torch.zeros(H, NB), v_scale=torch.zeros(H, NB))
    a.update(kw)
    return k.block_pool_q8_view(**a)


def views(k):
    return dict(pool=q8(k), pt=k.page_table_view(torch.zeros(B, MB, dtype=I32), torch.zeros(B, dtype=I32),
                                                 torch.zeros(B, dtype=I32), torch.zeros(B, MB)),
                free_pool=k.free_pool_view(torch.zeros(NB, dtype=I32), torch.zeros(1, dtype=I32)))


def ws():
    return torch.zeros(1 << 12, dtype=U8)


def norm_call(kvc, **kw):
    a = dict(q=torch.zeros(T, HQ, D), k=torch.zeros(T, H, D), w_q=torch.zeros(D), w_k=torch.zeros(D),
             cos_sin=torch.zeros(7, 2, 16), pos=torch.zeros(T, dtype=I32), q_out=torch.zeros(T, HQ, D),
             k_out=torch.zeros(T, H, D))
    a.update(kw)
    return kvc.kvc_qk_norm_rope(a.pop("q"), a.pop("k"), **a)


def append_call(k, **kw):
    a = dict(views(k), k_new=torch.zeros(T, H, D), v_new=torch.zeros(T, H, D), cu=torch.zeros(B + 1, dtype=I32),
             appended=torch.zeros(B, dtype=I32), ws=ws())
    a.update(kw)
    return k.kvc_paged_append_q8(*[a.pop(x) for x in ("pool", "pt", "free_pool", "k_new", "v_new")], **a)


def decode_call(k, **kw):
    v = views(k)
    a = dict(pool=v["pool"], pt=v["pt"], q=torch.zeros(B, HQ, D), scale=1.0, out=torch.zeros(B, HQ, D),
             logits=torch.zeros(B, HQ, MB * BS), lse=torch.zeros(B, HQ), ws=ws())
    a.update(kw)
    return k.kvc_decode_attn_paged_q8(a.pop("q"), a.pop("pool"), a.pop("pt"), **a)


def reorder_call(k, **kw):
    a = dict(views(k), shares=torch.zeros(NB, dtype=I32), parent=torch.zeros(B, dtype=I32),
             pos=torch.zeros(NB, BS, dtype=I32), ws=ws())
    a.update(kw)
    return k.kvc_pages_reorder(*[a.pop(x) for x in ("pool", "pt", "free_pool", "shares", "parent")], **a)


def compact_call(k, **kw):
    a = dict(views(k), shares=torch.zeros(NB, dtype=I32), pos=torch.zeros(NB, BS, dtype=I32),
             remap=torch.zeros(NB, dtype=I32), ws=ws())
    a.update(kw)
    return k.kvc_pages_compact(*[a.pop(x) for x in ("pool", "pt", "free_pool")], **a)


def wrong(t):
    """The same tensor with another type, shape, layout or device."""
    yield t.to({I32: torch.int64, F32: torch.float64}[t.dtype])
    yield torch.zeros((t.shape[0] + 1,) + t.shape[1:], dtype=t.dtype)
    yield torch.zeros(t.shape + (2,), dtype=t.dtype)[..., 0]
    yield Elsewhere(t)


@pytest.mark.parametrize("call,what,good", [
    (norm_call, "w_q", torch.zeros(D)), (norm_call, "w_k", torch.zeros(D)), (norm_call, "pos", torch.zeros(T, dtype=I32)),
    (append_call, "cu", torch.zeros(B + 1, dtype=I32)), (append_call, "appended", torch.zeros(B, dtype=I32)),
    (decode_call, "out", torch.zeros(B, HQ, D)), (decode_call, "logits", torch.zeros(B, HQ, MB * BS)),
    (decode_call, "lse", torch.zeros(B, HQ)), (reorder_call, "shares", torch.zeros(NB, dtype=I32)),
    (reorder_call, "parent", torch.zeros(B, dtype=I32)), (reorder_call, "pos", torch.zeros(NB, BS, dtype=I32)),
    (compact_call, "shares", torch.zeros(NB, dtype=I32)), (compact_call, "pos", torch.zeros(NB, BS, dtype=I32)),
    (compact_call, "remap", torch.zeros(NB, dtype=I32)),
])
def test_refused_by_name(kvc, call, what, good):
    call(kvc, **{what: good})
    assert len(kvc.stub_calls) == 1
    for bad in wrong(good):
        with pytest.raises(ValueError, match=f"^{what} must be"):
            call(kvc, **{what: bad})
    assert len(kvc.stub_calls) == 1


@pytest.mark.parametrize("call", [append_call, decode_call, reorder_call, compact_call])
def test_a_workspace_elsewhere_or_with_holes_is_refused(kvc, call):
    call(kvc)
    call(kvc, ws=OnDevice(-1))
    for bad in (OnDevice(0), OnDevice(-1, contiguous=False), torch.zeros(2048, dtype=U8)[::2]):
        with pytest.raises(ValueError, match="ws must be"):
            call(kvc, ws=bad)
    assert len(kvc.stub_calls) == 2


@pytest.mark.parametrize("call,names", [(append_call, ["pool", "pt", "free_pool"]), (decode_call, ["pool", "pt"]),
                                        (reorder_call, ["pt", "free_pool"]), (compact_call, ["pt", "free_pool"])])
def test_descriptors_with_a_tensor_elsewhere_are_refused(kvc, call, names):
    for what in names:
        view = views(kvc)[what]
        call(kvc, **{what: view})
        kept = view._keep
        for i in range(len(kept)):
            view._keep = kept[:i] + (Elsewhere(torch.zeros(1)),) + kept[i + 1:]
            with pytest.raises(ValueError, match=f"tensor of its {type(view).__name__}"):
                call(kvc, **{what: view})
    assert len(kvc.stub_calls) == len(names)


def test_rows_are_refused(kvc):
    q, k = torch.zeros(T, HQ, D), torch.zeros(T, H, D)
    away = Elsewhere(k)
    away.stride = k.stride
    for kw in (dict(q=q[0]), dict(k=k[:-1]), dict(k=k[..., :32]), dict(k=k.double()), dict(q=torch.zeros(T, HQ, D, 2)[..., 0]),
               dict(k=away), dict(k_out=away), dict(q_out=q[:, 1:]), dict(k_out=k[:, :1]), dict(q_out=q.to(BF16)),
               dict(cos_sin=None), dict(pos=None), dict(cos_sin=torch.zeros(7, 32))):
        with pytest.raises(ValueError):
            norm_call(kvc, **kw)
    with pytest.raises(TypeError):
        norm_call(kvc, q=q.double())
    for kw in (dict(k_new=k[:, :1]), dict(k_new=k[0]), dict(v_new=k[:, :1]), dict(v_new=k[:-1]), dict(v_new=away), dict(v_new=k.to(BF16)),
               dict(v_new=torch.zeros(T, H + 1, D)[:, :H]), dict(cu=None)):
        with pytest.raises(ValueError):
            append_call(kvc, **kw)
    with pytest.raises(TypeError):
        append_call(kvc, k_new=k.double())
    for kw in (dict(q=torch.zeros(B + 1, HQ, D)), dict(q=torch.zeros(B, HQ, 2 * D)), dict(q=torch.zeros(B, HQ * D)),
               dict(q=torch.zeros(HQ, B, D).transpose(0, 1)), dict(out=torch.zeros(B, HQ, D, dtype=BF16))):
        with pytest.raises(ValueError):
            decode_call(kvc, **kw)
    with pytest.raises(TypeError):
        decode_call(kvc, q=torch.zeros(B, HQ, D).double())
    with pytest.raises(ValueError, match="shares is needed"):
        reorder_call(kvc, shares=None)
    assert not kvc.stub_calls


def test_pools_are_refused(kvc):
    q8(kvc)
    q8(kvc, k_pool=torch.zeros(H, NB, BS, D).to(torch.float8_e4m3fn), v_pool=torch.zeros(H, NB, BS, D).to(torch.float8_e4m3fn))
    z = torch.zeros(H, NB, BS, D, dtype=U8)
    for kw in (dict(k_pool=z.to(torch.int8)), dict(k_pool=z[0]), dict(v_pool=z[:, :-1]), dict(v_pool=z.to(torch.float8_e4m3fn)),
               dict(v_pool=torch.zeros(H, NB, BS, 2 * D, dtype=U8)[..., ::2]), dict(k_scale=torch.zeros(H, NB + 1)),
               dict(v_scale=torch.zeros(H, NB, dtype=BF16)), dict(v_scale=torch.zeros(NB, H).T)):
        with pytest.raises(ValueError):
            q8(kvc, **kw)


def test_what_the_calls_make_themselves(kvc):
    """Workspaces and outputs that are not given, and calls without the arguments that may be left out."""
    a, b = norm_call(kvc, q_out=None, k_out=None)
    assert a.shape == (T, HQ, D) and b.shape == (T, H, D)
    norm_call(kvc, cos_sin=None, pos=None, w_k=None)
    append_call(kvc, ws=None, cu=None, appended=None, k_new=torch.zeros(B, H, D), v_new=torch.zeros(B, H, D))
    assert decode_call(kvc, ws=None, out=None, logits=None, lse=None).shape == (B, HQ, D)
    reorder_call(kvc, ws=None, pos=None, pool=kvc.block_pool_view(*[torch.zeros(H, NB, BS, D)] * 2))
    assert compact_call(kvc, ws=None, pos=None, shares=None, remap=None).shape == (NB,)
    assert len(kvc.stub_calls) == 6
