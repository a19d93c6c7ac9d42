"""What the binding of the draft-tree and latent calls checks, argument by argument: each wrong one is
refused by name, and a sound call gets through to the library.  On the CPU: the library is
replaced, and of the check for the current device, which no CPU tensor passes, only the part that
holds the descriptors' tensors against the call's device is left."""
import pytest
import torch

I32, I64, F32, BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16
B, HQ, H, D, T, CAP, BS, R, E = 2, 4, 2, 64, 4, 16, 8, 128, 64


class Lib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            if not name.endswith("workspace_bytes"):
                self.calls.append(name)
                return 0
            return 64
        return entry


class OnDevice:
    """A workspace as the binding sees it, on some device."""

    def __init__(self, index, contiguous=True):
        self.device, self.contiguous = f"cuda:{index}", contiguous
        self.get_device = lambda: index
        self.is_contiguous = lambda: self.contiguous
        self.data_ptr = lambda: 4096
        self.numel, self.element_size = (lambda: 1 << 20), (lambda: 1)
        self.dtype, self.shape = torch.uint8, (1 << 20,)


@pytest.fixture
def kvc(monkeypatch):
    from kv_cache_compression_kvc_gb300 import kvc as k
    lib = Lib()
    monkeypatch.setattr(k, "_lib", lib)
    monkeypatch.setattr(k, "load", lambda: lib)
    monkeypatch.setattr(k, "_on_current", k._beside)
    monkeypatch.setattr(k, "_raw_stream", lambda *a: 0)
    k.stub_calls = lib.calls
    yield k
    del k.stub_calls


def tree_call(k, **kw):
    a = dict(q=torch.zeros(B, T, HQ, D), cache=k.cache_view(torch.zeros(B, H, CAP, D), torch.zeros(B, H, CAP, D)),
             draft=k.make_draft(torch.zeros(B, T, H, D), torch.zeros(B, T, H, D)), scale=1.0,
             len=torch.zeros(B, H, dtype=I32), lse=torch.zeros(B, T, HQ), out=torch.zeros(B, T, HQ, D),
             ws=torch.zeros(1024, dtype=torch.uint8))
    a.update(kw)
    return k.kvc_decode_attn_tree(a.pop("q"), a.pop("cache"), a.pop("draft"), **a)


def paged_call(k, **kw):
    a = dict(q=torch.zeros(B, T, HQ, D), pool=k.block_pool_view(torch.zeros(H, 9, BS, D), torch.zeros(H, 9, BS, D)),
             pt=k.page_table_view(torch.zeros(B, 2, dtype=I32), torch.zeros(B, dtype=I32),
                                  torch.zeros(B, dtype=I32), torch.zeros(B, 2)),
             draft=k.make_draft(torch.zeros(B, T, H, D), torch.zeros(B, T, H, D)), scale=1.0,
             lse=torch.zeros(B, T, HQ), out=torch.zeros(B, T, HQ, D), ws=torch.zeros(1024, dtype=torch.uint8))
    a.update(kw)
    return k.kvc_decode_attn_tree_paged(a.pop("q"), a.pop("pool"), a.pop("pt"), a.pop("draft"), **a)


def latent_call(k, **kw):
    a = dict(q=torch.zeros(B, T, HQ, R + E), cache=k.latent_cache_view(torch.zeros(B, CAP, R + E), R),
             draft=k.make_draft(torch.zeros(B, T, R + E)), scale=1.0, len=torch.zeros(B, dtype=I32),
             lse=torch.zeros(B, T, HQ), out=torch.zeros(B, T, HQ, R), ws=torch.zeros(1024, dtype=torch.uint8))
    a.update(kw)
    return k.kvc_decode_attn_latent(a.pop("q"), a.pop("cache"), a.pop("draft"), **a)


CALLS = {"tree": tree_call, "paged": paged_call, "latent": latent_call}


@pytest.mark.parametrize("call", CALLS)
def test_a_workspace_elsewhere_or_with_holes_is_refused(kvc, call):
    """The kernels write to its address: it lies on their device, and its extent is its size."""
    fn = CALLS[call]
    fn(kvc)
    fn(kvc, ws=OnDevice(-1))
    assert len(kvc.stub_calls) == 2
    for ws in (OnDevice(0), OnDevice(1), OnDevice(-1, contiguous=False),
               torch.zeros(2048, dtype=torch.uint8)[::2], torch.zeros(1, dtype=torch.uint8).expand(4096)):
        with pytest.raises(ValueError, match="ws must be"):
            fn(kvc, ws=ws)
    assert len(kvc.stub_calls) == 2


class Elsewhere:
    """A tensor that is right but for its device."""

    def __init__(self, t, index=0):
        self.dtype, self.shape, self.device = t.dtype, t.shape, f"cuda:{index}"
        self.is_contiguous, self.get_device, self.data_ptr = (lambda: True), (lambda: index), (lambda: 4096)
        self.dim = t.dim


def wrong(t):
    """The same tensor with another type, shape, layout or device."""
    other = {I32: I64, F32: torch.float64}[t.dtype]
    yield t.to(other)
    yield torch.zeros(t.shape[:-1] + (t.shape[-1] + 1,), dtype=t.dtype)
    yield torch.zeros((t.shape[0] + 1,) + t.shape[1:], dtype=t.dtype)
    yield torch.zeros(t.shape + (2,), dtype=t.dtype)[..., 0]
    yield Elsewhere(t)


ATTENTION = [
    ("tree", "len", torch.zeros(B, H, dtype=I32)), ("tree", "lse", torch.zeros(B, T, HQ)),
    ("tree", "out", torch.zeros(B, T, HQ, D)), ("paged", "lse", torch.zeros(B, T, HQ)),
    ("paged", "out", torch.zeros(B, T, HQ, D)), ("latent", "len", torch.zeros(B, dtype=I32)),
    ("latent", "lse", torch.zeros(B, T, HQ)), ("latent", "out", torch.zeros(B, T, HQ, R)),
]


@pytest.mark.parametrize("call,what,good", ATTENTION)
def test_attention_refuses_by_name(kvc, call, what, good):
    CALLS[call](kvc, **{what: good})
    assert len(kvc.stub_calls) == 1
    for bad in wrong(good):
        with pytest.raises(ValueError, match=f"^{what} must be"):
            CALLS[call](kvc, **{what: bad})
    assert len(kvc.stub_calls) == 1


def test_attention_takes_lengths_in_one_row(kvc):
    tree_call(kvc, len=torch.zeros(B * H, dtype=I32))
    assert len(kvc.stub_calls) == 1
    with pytest.raises(ValueError, match="^len must be"):
        tree_call(kvc, len=torch.zeros(B, dtype=I32))


@pytest.mark.parametrize("call,q", [("tree", torch.zeros(B, T, HQ, D)), ("paged", torch.zeros(B, T, HQ, D)),
                                    ("latent", torch.zeros(B, T, HQ, R + E))])
def test_attention_refuses_queries(kvc, call, q):
    for bad in (q.double(), q[:, :3], q[:1], q[..., :-8].contiguous(), q[0], q.transpose(1, 2),
                torch.zeros(q.shape + (2,))[..., 0]):
        with pytest.raises(ValueError, match="^q must be"):
            CALLS[call](kvc, q=bad)
    assert not kvc.stub_calls


def drafts(k):
    """Drafts that are sound but not the cache's: type, batch, heads, width, latent or not."""
    yield k.make_draft(torch.zeros(B, T, H, D, dtype=BF16), torch.zeros(B, T, H, D, dtype=BF16))
    yield k.make_draft(torch.zeros(B + 1, T, H, D), torch.zeros(B + 1, T, H, D))
    yield k.make_draft(torch.zeros(B, T, H + 1, D), torch.zeros(B, T, H + 1, D))
    yield k.make_draft(torch.zeros(B, T, H, 2 * D), torch.zeros(B, T, H, 2 * D))
    yield k.make_draft(torch.zeros(B, T, R + E + 8))
    yield k.make_draft(torch.zeros(B, T, H * D))


def test_every_call_refuses_drafts_of_another_cache(kvc):
    for d in drafts(kvc):
        for call in (*CALLS.values(), accept_call, accept_paged_call, latent_accept_call):
            with pytest.raises(ValueError, match="^drafted rows must be"):
                call(kvc, draft=d)
    d = kvc.make_draft(n_draft=T)
    for call in CALLS.values():
        call(kvc, draft=d)                                    # the cache alone
    for call in (accept_call, accept_paged_call, latent_accept_call):
        with pytest.raises(ValueError, match="needs the drafted rows"):
            call(kvc, draft=d)
    assert len(kvc.stub_calls) == 3
    for call in CALLS.values():
        with pytest.raises(ValueError, match="^count must be"):
            call(kvc, draft=kvc.make_draft(n_draft=T, count=torch.zeros(B + 1, dtype=I32)))


def accept_call(k, **kw):
    a = dict(cache=k.cache_view(torch.zeros(B, H, CAP, D), torch.zeros(B, H, CAP, D)),
             len=torch.zeros(B, H, dtype=I32), draft=k.make_draft(torch.zeros(B, T, H, D), torch.zeros(B, T, H, D)),
             path=torch.zeros(B, T, dtype=I32), n_accept=torch.zeros(B, dtype=I32))
    a.update(kw)
    return k.kvc_tree_accept(**a)


def accept_paged_call(k, **kw):
    a = dict(pool=k.block_pool_view(torch.zeros(H, 9, BS, D), torch.zeros(H, 9, BS, D)),
             pt=k.page_table_view(torch.zeros(B, 2, dtype=I32), torch.zeros(B, dtype=I32),
                                  torch.zeros(B, dtype=I32), torch.zeros(B, 2)),
             free_pool=k.free_pool_view(torch.zeros(9, dtype=I32), torch.zeros(1, dtype=I32)),
             draft=k.make_draft(torch.zeros(B, T, H, D), torch.zeros(B, T, H, D)),
             path=torch.zeros(B, T, dtype=I32), n_accept=torch.zeros(B, dtype=I32),
             accepted=torch.zeros(B, dtype=I32))
    a.update(kw)
    return k.kvc_tree_accept_paged(**a)


def latent_accept_call(k, **kw):
    a = dict(cache=k.latent_cache_view(torch.zeros(B, CAP, R + E), R), len=torch.zeros(B, dtype=I32),
             draft=k.make_draft(torch.zeros(B, T, R + E)), path=torch.zeros(B, T, dtype=I32),
             n_accept=torch.zeros(B, dtype=I32))
    a.update(kw)
    return k.kvc_latent_accept(**a)


def expand_call(k, **kw):
    a = dict(cache=k.latent_cache_view(torch.zeros(B, CAP, 192), 128), w_k=torch.zeros(H, 64, 128),
             w_v=torch.zeros(H, 128, 128), dst=k.cache_view(torch.zeros(B, H, CAP, 128), torch.zeros(B, H, CAP, 128)),
             len=torch.zeros(B, dtype=I32))
    a.update(kw)
    return k.kvc_latent_expand(**a)


@pytest.mark.parametrize("call,what,good", [
    (accept_call, "len", torch.zeros(B, H, dtype=I32)), (accept_call, "path", torch.zeros(B, T, dtype=I32)),
    (accept_call, "n_accept", torch.zeros(B, dtype=I32)),
    (accept_paged_call, "path", torch.zeros(B, T, dtype=I32)),
    (accept_paged_call, "n_accept", torch.zeros(B, dtype=I32)),
    (accept_paged_call, "accepted", torch.zeros(B, dtype=I32)),
    (latent_accept_call, "len", torch.zeros(B, dtype=I32)),
    (latent_accept_call, "path", torch.zeros(B, T, dtype=I32)),
    (latent_accept_call, "n_accept", torch.zeros(B, dtype=I32)),
    (expand_call, "len", torch.zeros(B, dtype=I32)), (expand_call, "w_k", torch.zeros(H, 64, 128)),
    (expand_call, "w_v", torch.zeros(H, 128, 128)),
])
def test_accept_and_expand_refuse_by_name(kvc, call, what, good):
    call(kvc, **{what: good})
    assert len(kvc.stub_calls) == 1
    for bad in wrong(good):
        # (the device of w_k is the call's own: the descriptors' are held against it)
        own = what == "w_k" and isinstance(bad, Elsewhere)
        with pytest.raises(ValueError, match="^w_k is on" if own else f"^{what} must be"):
            call(kvc, **{what: bad})
    assert len(kvc.stub_calls) == 1


def test_a_draft_refuses_its_tensors(kvc):
    k, lat = torch.zeros(B, T, H, D), torch.zeros(B, T, R + E)
    for bad, match in [
        (dict(k=k), "need values"), (dict(k=lat, v=lat), "need values"), (dict(k=k[0, 0], v=k[0, 0]), "contiguous"),
        (dict(k=k.transpose(0, 1), v=k), "contiguous"), (dict(k=k, v=k.transpose(0, 1)), "match"),
        (dict(k=k, v=k.double()), "match"), (dict(k=k, v=k[:, :2]), "match"), (dict(k=k, v=k, n_draft=5), "n_draft 5"),
        (dict(v=k), "needs its keys"), (dict(), "needs its keys"),
        (dict(n_draft=T, mask=torch.zeros(B, T, dtype=I64)), "mask needs"),
        (dict(n_draft=T, count=torch.zeros(B, dtype=I64)), "count must be"),
        (dict(n_draft=T, count=torch.zeros(B, 2, dtype=I32)[:, 0]), "count must be"),
    ]:
        with pytest.raises(ValueError, match=match):
            kvc.make_draft(**bad)
    for what, good in (("mask", torch.zeros(B, T, dtype=I64)), ("count", torch.zeros(B, dtype=I32))):
        kvc.make_draft(k, k, **{what: good})
        kvc.make_draft(lat, **{what: good})
        for bad in (good.float(), torch.zeros(good.shape + (2,), dtype=good.dtype)[..., 0], good[:1], Elsewhere(good)):
            with pytest.raises(ValueError, match=f"^{what} must be"):
                kvc.make_draft(k, k, **{what: bad})


@pytest.mark.parametrize("call,views", [
    (tree_call, ["cache"]), (paged_call, ["pool", "pt"]), (latent_call, ["cache"]), (accept_call, ["cache"]),
    (accept_paged_call, ["pool", "pt", "free_pool"]), (latent_accept_call, ["cache"]), (expand_call, ["cache", "dst"]),
])
def test_descriptors_with_a_tensor_elsewhere_are_refused(kvc, call, views):
    made = {"cache": lambda: (kvc.latent_cache_view(torch.zeros(B, CAP, R + E), R)
                              if call in (latent_call, latent_accept_call, expand_call) else
                              kvc.cache_view(torch.zeros(B, H, CAP, D), torch.zeros(B, H, CAP, D))),
            "pool": lambda: kvc.block_pool_view(torch.zeros(H, 9, BS, D), torch.zeros(H, 9, BS, D)),
            "pt": lambda: kvc.page_table_view(torch.zeros(B, 2, dtype=I32), torch.zeros(B, dtype=I32),
                                              torch.zeros(B, dtype=I32), torch.zeros(B, 2)),
            "free_pool": lambda: kvc.free_pool_view(torch.zeros(9, dtype=I32), torch.zeros(1, dtype=I32)),
            "dst": lambda: kvc.cache_view(torch.zeros(B, H, CAP, 128), torch.zeros(B, H, CAP, 128))}
    for what in views:
        view = made[what]()
        call(kvc, **{what: view})
        kept = view._keep if type(view._keep) is tuple else (view._keep,)
        for i in range(len(kept)):
            view._keep = kept[:i] + (Elsewhere(torch.zeros(1)),) + kept[i + 1:]
            with pytest.raises(ValueError, match=f"tensor of its {type(view).__name__}"):
                call(kvc, **{what: view})
    assert len(kvc.stub_calls) == len(views)
