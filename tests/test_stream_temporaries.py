"""What a call makes for itself (outputs, workspaces) it makes on the stream that its kernels run on:
torch's allocator hands a freed tensor's memory on in the order of the stream that it was made on, so a
workspace of the current stream, freed when the call returns, could be another tensor's while kernels
on `stream` still use it.  On the CPU, with the library and the streams replaced."""
import contextlib

import pytest
import torch


class Stream:
    cuda_stream = 7


class Lib:
    """Every entry point succeeds; every workspace query asks for 64 bytes."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            if name.endswith("workspace_bytes"):
                return 64
            self.calls.append((name, args))
            return 0
        return entry


B, HQ, H, D, T, CAP, BS = 2, 4, 2, 64, 3, 16, 8
I32 = torch.int32


def caches(heads=H):
    return torch.zeros(B, heads, CAP, D), torch.zeros(B, heads, CAP, D)


def pages(kvc):
    pool = kvc.block_pool_view(torch.zeros(H, 9, BS, D), torch.zeros(H, 9, BS, D))
    pt = kvc.page_table_view(torch.zeros(B, 2, dtype=I32), torch.zeros(B, dtype=I32), torch.zeros(B, dtype=I32),
                             torch.zeros(B, 2))
    return pool, pt, kvc.free_pool_view(torch.zeros(9, dtype=I32), torch.zeros(1, dtype=I32))


def tree_draft(kvc):
    return kvc.make_draft(torch.zeros(B, T, H, D), torch.zeros(B, T, H, D))


def duo(kvc):
    full, ring = (kvc.cache_view(*caches(1)) for _ in range(2))
    return full, ring, kvc.Duo([0], 4, 8, torch.zeros(1, dtype=torch.int64))


Q, QT = torch.zeros(B, HQ, D), torch.zeros(B, T, HQ, D)
CALLS = {
    "kvc_decode_attn": lambda k, s: k.kvc_decode_attn(Q, *caches(), scale=1.0, n_valid=4, stream=s),
    "kvc_decode_attn_ex": lambda k, s: k.kvc_decode_attn_ex(Q, *caches(), scale=1.0, n_valid=4, stream=s),
    "kvc_decode_attn_alibi": lambda k, s: k.kvc_decode_attn_alibi(
        Q, *caches(), scale=1.0, alibi=k.make_alibi(4, 8, torch.zeros(1, dtype=torch.int64), torch.zeros(HQ)), stream=s),
    "kvc_decode_attn_paged": lambda k, s: k.kvc_decode_attn_paged(Q, *pages(k)[:2], scale=1.0, stream=s),
    "kvc_decode_attn_duo": lambda k, s: k.kvc_decode_attn_duo(Q, *duo(k), scale=1.0, n_valid=4, stream=s),
    "kvc_decode_attn_noalloc": lambda k, s: k.kvc_decode_attn_noalloc(Q, *caches(), scale=1.0, n_valid=4, stream=s),
    "kvc_block_prompt_select": lambda k, s: k.kvc_block_prompt_select(
        torch.zeros(B, H, CAP), *caches(), *pages(k), seq_len=CAP, budget_blocks=2, recent_blocks=1, stream=s),
    "kvc_snapkv_select": lambda k, s: k.kvc_snapkv_select(
        torch.zeros(B, HQ, 4, D), caches()[0], seq_len=CAP, L_obs=4, budget=8, scale=1.0, stream=s),
    "kvc_h2o_prefill_select": lambda k, s: k.kvc_h2o_prefill_select(
        torch.zeros(B, H, CAP, D), caches()[0], seq_len=CAP, L_local=4, K_hh=4, scale=1.0, stream=s),
    "kvc_h2o_prefill_select_gqa": lambda k, s: k.kvc_h2o_prefill_select_gqa(
        torch.zeros(B, HQ, CAP, D), caches()[0], seq_len=CAP, L_local=4, K_hh=4, scale=1.0, stream=s),
    "kvc_decode_attn_tree": lambda k, s: k.kvc_decode_attn_tree(
        QT, k.cache_view(*caches()), tree_draft(k), scale=1.0, n_valid=4, stream=s),
    "kvc_decode_attn_tree_paged": lambda k, s: k.kvc_decode_attn_tree_paged(
        QT, *pages(k)[:2], tree_draft(k), scale=1.0, stream=s),
    "kvc_decode_attn_latent": lambda k, s: k.kvc_decode_attn_latent(
        torch.zeros(B, T, HQ, 192), k.latent_cache_view(torch.zeros(B, CAP, 192), 128),
        k.make_draft(torch.zeros(B, T, 192)), scale=1.0, n_valid=4, stream=s),
    "kvc_tree_accept_paged": lambda k, s: k.kvc_tree_accept_paged(
        *pages(k), tree_draft(k), torch.zeros(B, T, dtype=I32), torch.zeros(B, dtype=I32), stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_call_makes_its_tensors_on_its_stream(name, monkeypatch):
    from kv_cache_compression_kvc_gb300 import kvc
    lib = Lib()
    monkeypatch.setattr(kvc, "_lib", lib)
    monkeypatch.setattr(kvc, "load", lambda: lib)
    monkeypatch.setattr(kvc, "_on_current", lambda *a: None)
    current, made = [None], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)

    def watch(fn):
        def make(*args, **kw):
            made.append(current[-1])
            return fn(*args, **kw)
        return make

    stream = Stream()
    own = []                                   # what building the arguments makes does not count
    real = {f: getattr(torch, f) for f in ("empty", "zeros", "empty_like", "full")}
    call = getattr(kvc, name)

    def entered(*args, **kw):
        with monkeypatch.context() as m:
            for f, fn in real.items():
                m.setattr(torch, f, watch(fn))
            out = call(*args, **kw)
        own.extend(made)
        return out

    monkeypatch.setattr(kvc, name, entered)
    CALLS[name](kvc, stream)
    assert [n for n, _ in lib.calls] == [name] and current == [None]
    assert own and all(s is stream for s in own), f"{own.count(None)} of {len(own)} on the current stream"
