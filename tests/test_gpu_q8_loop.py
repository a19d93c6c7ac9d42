"""The operators together, as serving uses them: norms and rotation, rows into 8-bit pages, attention over
them, block eviction by its logits; beams that share pages; and the binding's own workspaces."""
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


def make(kvc, B, H, D, bs, NB, mb):
    s = dict(k=torch.zeros((H, NB, bs, D), dtype=torch.uint8, device=DEV), v=torch.zeros((H, NB, bs, D), dtype=torch.uint8, device=DEV),
             ks=torch.zeros((H, NB), device=DEV), vs=torch.zeros((H, NB), device=DEV),
             table=torch.zeros((B, mb), dtype=torch.int32, device=DEV), n_blocks=torch.zeros(B, dtype=torch.int32, device=DEV),
             len=torch.zeros(B, dtype=torch.int32, device=DEV), score=torch.zeros((B, mb), device=DEV),
             ids=torch.arange(NB, dtype=torch.int32, device=DEV), top=torch.tensor([NB], dtype=torch.int32, device=DEV))
    s["pool"] = kvc.block_pool_q8_view(s["k"], s["v"], s["ks"], s["vs"])
    s["pt"] = kvc.page_table_view(s["table"], s["n_blocks"], s["len"], s["score"])
    s["free"] = kvc.free_pool_view(s["ids"], s["top"])
    return s


def dequantised(s, b, h, bs):
    n = int(s["len"][b])
    t = s["table"][b, : (n + bs - 1) // bs].long()
    return [(s[x][h, t].view(torch.float8_e4m3fn).double() * s[x + "s"][h, t].double()[:, None, None]).flatten(0, 1)[:n]
            for x in "kv"]


def rows(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def same(out, q, s, b, H, G, bs, scale):
    """bf16 outputs: 2^-8 of the value, 2^-11 of the weights and some 2^-14 for fp32 logits of size 10."""
    for h in range(H):
        k, v = dequantised(s, b, h, bs)
        want, _, _, size = attention(q[b, h * G:(h + 1) * G].double(), k, v, scale)
        got = out[b, h * G:(h + 1) * G].double()
        assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -14) * size + 1e-12).all())


def test_prompt_then_decode_with_eviction(kvc):
    """Prompts of different lengths, then steps; what the pages hold stays near the rows that went in."""
    B, Hq, H, D, bs, mb = 3, 8, 2, 64, 16, 8
    G, scale = Hq // H, 1.0 / math.sqrt(D)
    s = make(kvc, B, H, D, bs, 40, mb)
    cs = kvc.kvc_rope_table(512, D).to(DEV)
    wq, wk = rows(1, D), rows(2, D)
    lens = [37, 1, 80]
    cu = torch.tensor([0, 37, 38, 118], dtype=torch.int32, device=DEV)
    qkv = rows(3, 118, Hq + 2 * H, D)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).to(DEV)
    _, k = kvc.kvc_qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + H], w_q=wq, w_k=wk, cos_sin=cs, pos=pos)
    v = qkv[:, Hq + H:].contiguous()
    kvc.kvc_paged_append_q8(s["pool"], s["pt"], s["free"], k, v, cu=cu)
    for b, n in enumerate(lens):
        for h in range(H):
            for got, want in zip(dequantised(s, b, h, bs), (k, v)):
                want = want[int(cu[b]):int(cu[b]) + n, h].double()
                # half a step of 4 significant bits, and of the smallest step of a page
                assert bool(((got - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -17 * want.abs().max()).all())
    for step in range(60):
        qkv = rows(100 + step, B, Hq + 2 * H, D)
        pos = s["len"].clone()
        q, k = kvc.kvc_qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + H], w_q=wq, w_k=wk, cos_sin=cs, pos=pos)
        kvc.kvc_paged_append_q8(s["pool"], s["pt"], s["free"], k, qkv[:, Hq + H:].contiguous())
        logits = torch.zeros((B, Hq, mb * bs), device=DEV)
        lse = torch.empty((B, Hq), device=DEV)
        out = kvc.kvc_decode_attn_paged_q8(q, s["pool"], s["pt"], scale=scale, logits=logits, lse=lse)
        if step % 13 == 0:
            for b in range(B):
                same(out, q, s, b, H, G, bs, scale)
        before = s["score"].clone(), s["n_blocks"].clone(), s["len"].clone()
        kvc.kvc_block_accumulate_evict(logits, lse, s["pt"], s["free"], block_size=bs, budget_blocks=5, recent_blocks=2)
        assert bool((s["n_blocks"] <= 5).all())
        for b in range(B):                       # every step spreads one unit of attention a query head
            if int(s["n_blocks"][b]) == int(before[1][b]):
                gain = float((s["score"][b] - before[0][b])[: int(before[1][b])].sum())
                assert abs(gain - Hq) < 1e-3
    assert kvc.kvc_device_status() == 0


def test_beams_over_8_bit_pages(kvc):
    """One prompt, four beams: forked, decoded, reordered and compacted; every beam attends to its own rows."""
    B, Hq, H, D, bs, mb = 4, 6, 1, 128, 16, 10
    scale = 1.0 / math.sqrt(D)
    s = make(kvc, B, H, D, bs, 60, mb)
    shares = torch.zeros(60, dtype=torch.int32, device=DEV)
    par = lambda *p: torch.tensor(p, dtype=torch.int32, device=DEV)  # noqa: E731
    prompt = rows(1, 45, H, D)
    kvc.kvc_paged_append_q8(s["pool"], s["pt"], s["free"], prompt, -prompt, cu=par(0, 45, 45, 45, 45))
    kvc.kvc_pages_reorder(s["pool"], s["pt"], s["free"], shares, par(0, 0, 0, 0))
    assert int(s["top"]) == 60 - 2 - 4           # two full pages shared, a partly filled one each
    parents = [(0, 0, 1, 3), (2, 1, 1, 0), (3, 3, 3, 3), (0, 1, 2, 3)]
    for step in range(24):
        k = rows(10 + step, B, H, D)
        kvc.kvc_paged_append_q8(s["pool"], s["pt"], s["free"], k, k)
        q = rows(50 + step, B, Hq, D)
        out = kvc.kvc_decode_attn_paged_q8(q, s["pool"], s["pt"], scale=scale)
        for b in range(B):
            same(out, q, s, b, H, Hq, bs, scale)
        held = [dequantised(s, b, 0, bs) for b in range(B)]
        p = parents[step % 4]
        kvc.kvc_pages_reorder(s["pool"], s["pt"], s["free"], shares, par(*p))
        if step % 5 == 4:
            kvc.kvc_pages_compact(s["pool"], s["pt"], s["free"], shares=shares)
        for b in range(B):
            for got, want in zip(dequantised(s, b, 0, bs), held[p[b]]):
                assert torch.equal(got, want)
    kvc.kvc_pages_reorder(s["pool"], s["pt"], s["free"], shares, par(-1, -1, -1, -1))
    assert int(s["top"]) == 60 and not bool(shares.any()) and kvc.kvc_device_status() == 0


def test_a_captured_step_is_an_eager_one(kvc):
    """Norms, append, attention, eviction and a reorder captured once and replayed, against the same calls."""
    B, Hq, H, D, bs, mb, NB = 3, 8, 2, 64, 16, 6, 40
    cs = kvc.kvc_rope_table(256, D).to(DEV)
    w = rows(1, D)
    runs = []
    for captured in (False, True):
        s = make(kvc, B, H, D, bs, NB, mb)
        shares = torch.zeros(NB, dtype=torch.int32, device=DEV)
        par = torch.tensor([2, 1, 0], dtype=torch.int32, device=DEV)
        qkv, lse = torch.zeros((B, Hq + 2 * H, D), dtype=torch.bfloat16, device=DEV), torch.zeros((B, Hq), device=DEV)
        logits, out = torch.zeros((B, Hq, mb * bs), device=DEV), torch.zeros((B, Hq, D), dtype=torch.bfloat16, device=DEV)
        qo, ko = torch.zeros_like(out), torch.zeros((B, H, D), dtype=torch.bfloat16, device=DEV)
        v = torch.zeros((B, H, D), dtype=torch.bfloat16, device=DEV)
        spaces = (kvc.append_q8_workspace(B, B, bs, DEV), kvc.decode_q8_workspace(B, Hq, H, D, torch.bfloat16, DEV),
                  kvc.pages_workspace(B, mb, NB, DEV))

        def step():
            kvc.kvc_qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + H], w_q=w, w_k=w, cos_sin=cs, pos=s["len"], q_out=qo, k_out=ko)
            v.copy_(qkv[:, Hq + H:])
            kvc.kvc_paged_append_q8(s["pool"], s["pt"], s["free"], ko, v, ws=spaces[0])
            kvc.kvc_decode_attn_paged_q8(qo, s["pool"], s["pt"], scale=0.125, out=out, logits=logits, lse=lse, ws=spaces[1])
            kvc.kvc_block_accumulate_evict(logits, lse, s["pt"], s["free"], block_size=bs, budget_blocks=4, recent_blocks=2)
            kvc.kvc_pages_reorder(s["pool"], s["pt"], s["free"], shares, par, ws=spaces[2])

        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        outs = []
        for i in range(90):
            qkv.copy_(rows(100 + i, B, Hq + 2 * H, D))
            graph.replay() if captured else step()
            outs.append(out.clone())
        assert kvc.kvc_device_status() == 0 and not bool(shares.any())
        runs.append((torch.stack(outs), s["len"].clone(), s["n_blocks"].clone(), s["score"].clone()))
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_two_streams_with_workspaces_of_their_own(kvc):
    """Two calls at once on different streams, each with a workspace that the binding made."""
    B, H, D, bs = 2, 2, 64, 16
    a, b = make(kvc, B, H, D, bs, 200, 64), make(kvc, B, H, D, bs, 200, 64)
    x = rows(5, 2 * 900, H, D)
    cu = torch.tensor([0, 900, 1800], dtype=torch.int32, device=DEV)
    q = rows(6, B, 8, D)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for s, st, y in ((a, streams[0], x), (b, streams[1], -x)):
        kvc.kvc_paged_append_q8(s["pool"], s["pt"], s["free"], y, x, cu=cu, stream=st)
        outs.append(kvc.kvc_decode_attn_paged_q8(q, s["pool"], s["pt"], scale=0.1, stream=st))
    torch.cuda.synchronize()
    for s, out in zip((a, b), outs):
        for i in range(B):
            same(out, q, s, i, H, 4, bs, 0.1)
