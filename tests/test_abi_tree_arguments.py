"""What the binding of the draft-tree and latent calls checks, argument by argument: each wrong one is
refused by name, and a sound call gets through to the library.  On the CPU: the library is
replaced, and the check for the current device, which no CPU tensor passes, is left out."""
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
    monkeypatch.setattr(k, "_on_current", lambda *a: None)
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
