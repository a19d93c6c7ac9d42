"""Measured cases of the operators around a paged cache: norms and rotation of queries and keys,
pages held in 8 bits (append and attention), pages shared between sequences, pools made dense.

Each case is one pass through one operator.  With ``own`` false the pass is made of elementary
torch operations in fp32; with ``own`` true it is the call a user of the library makes.
"""
import math

import torch

own = False

# --------------------------------------------------------------------------------------------
# Cases.  op: "norm" (RMS norm of every query and key head, then the rotation to the token's
# position), "append" (new rows into pages of e4m3 numbers with a scale for each page and head),
# "decode" (attention of one new token per sequence over such pages), "reorder" (every sequence
# becomes a copy of another one or is freed, full pages shared), "compact" (the pool's live pages
# move to its lowest ids).  Lengths run evenly from lo to hi over the sequences.


def listed():
    return [
        # one decode step of 16 sequences, 32 query and 32 key heads: latency of one call
        dict(name="norm_step", op="norm", dtype="bf16", T=16, Hq=32, Hkv=32, D=128, rot=128, n_pos=8192),
        # a 32768-token prompt of the grouped workload: every query and key once through HBM
        dict(name="norm_prompt", op="norm", dtype="bf16", T=32768, Hq=32, Hkv=8, D=128, rot=128, n_pos=32768),
        # one new token for each of 16 sequences of the block-eviction workload: latency
        dict(name="append_step", op="append", dtype="bf16", B=16, Hkv=32, D=128, bs=32, lo=801, hi=832, new_lo=1, new_hi=1),
        # 16 prompts of 2048 to 4096 tokens, 32 heads: rows in, 8-bit pages out
        dict(name="append_prompts", op="append", dtype="bf16", B=16, Hkv=32, D=128, bs=32, lo=0, hi=0, new_lo=2048, new_hi=4096),
        # a short prompt of the small test workload: latency of one call
        dict(name="decode_small", op="decode", dtype="bf16", B=1, Hq=8, Hkv=2, D=64, bs=16, lo=128, hi=128),
        # the block-eviction workload: 512 rows of 26 pages, one query head per KV head
        dict(name="decode_blocks", op="decode", dtype="bf16", B=16, Hq=32, Hkv=32, D=128, bs=32, lo=801, hi=832),
        # uncompressed 128k-token caches of the grouped workload: the most bytes per call
        dict(name="decode_long", op="decode", dtype="bf16", B=2, Hq=32, Hkv=8, D=128, bs=32, lo=131072, hi=131072),
        # pyramid budgets (four to one over the sequences), fp32 queries, d_head 256, groups of six
        dict(name="decode_pyramid", op="decode", dtype="fp32", B=8, Hq=24, Hkv=4, D=256, bs=16, lo=3277, hi=13107),
        # four beams of one short prompt, fp32: latency of one call
        dict(name="reorder_small", op="reorder", dtype="fp32", B=4, group=4, Hkv=2, D=64, bs=16, lo=100, hi=128),
        # 16 prompts with 8 beams each, pages of 32 tokens and 32 heads
        dict(name="reorder_beams", op="reorder", dtype="bf16", B=128, group=8, Hkv=32, D=128, bs=32, lo=801, hi=832),
        # a small pool, half of it live: latency of one call
        dict(name="compact_small", op="compact", dtype="bf16", NB=64, live=50, Hkv=2, D=64, bs=16),
        # a pool of 524288 tokens in 8 bits, 60 per cent live after long serving
        dict(name="compact_large", op="compact", dtype="e4m3", NB=16384, live=60, Hkv=8, D=128, bs=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges; costs no more than the largest listed one."""
    op = rng.choice(["norm", "append", "append", "decode", "decode", "decode", "reorder", "compact"])
    dt = rng.choice(["bf16", "bf16", "fp32"])
    D = rng.choice([64, 128, 256])
    if op == "norm":
        c = dict(op=op, dtype=dt, Hkv=rng.choice([1, 2, 3, 8, 32]), D=D, rot=rng.choice([0, D // 4, D // 2, D, D]),
                 n_pos=_log(rng, 64, 131072))
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 4, 6])
        limit = 2 ** 27 if dt == "bf16" else 2 ** 26                     # elements
        c["T"] = max(1, min(_log(rng, 1, 65536), limit // ((c["Hq"] + c["Hkv"]) * D)))
        return c
    H = rng.choice([1, 2, 3, 4, 8, 16, 32])
    bs = rng.choice([16, 32, 64])
    if op == "append":
        c = dict(op=op, dtype=dt, B=_log(rng, 1, 64), Hkv=H, D=D, bs=bs)
        limit = 2 ** 27 if dt == "bf16" else 2 ** 26                     # elements of new keys
        hi = _log(rng, 1, 8192) if rng.random() < 0.6 else 1
        hi = max(1, min(hi, limit // (c["B"] * H * D)))
        c["new_hi"], c["new_lo"] = hi, rng.randint(1, hi)
        c["hi"] = rng.randint(0, 900)
        c["lo"] = rng.randint(0, c["hi"])
        return c
    if op == "decode":
        c = dict(op=op, dtype=dt, B=_log(rng, 1, 64), Hkv=H, D=D, bs=bs)
        c["Hq"] = H * rng.choice([1, 2, 4, 6, 8, 12])
        hi = _log(rng, 8, 131072) if rng.random() < 0.9 else rng.randint(0, 3)
        limit = 2 ** 27 if dt == "bf16" else 2 ** 26                     # elements of keys
        hi = max(1, min(hi, limit // (c["B"] * H * D)))
        c["hi"], c["lo"] = hi, rng.randint(0, hi)
        return c
    dt = rng.choice(["bf16", "bf16", "fp32", "e4m3"])
    if op == "reorder":
        g = rng.choice([1, 2, 4, 5, 8])
        c = dict(op=op, dtype=dt, B=g * _log(rng, 1, 32), group=g, Hkv=H, D=D, bs=bs)
        page = H * D * bs * {"bf16": 2, "fp32": 4, "e4m3": 1}[dt]
        hi = max(1, min(_log(rng, 1, 4096), 2 ** 29 // (page * c["B"]) * bs))
        c["hi"], c["lo"] = hi, rng.randint(0, hi)
        return c
    page = H * D * bs * {"bf16": 2, "fp32": 4, "e4m3": 1}[dt]
    nb = max(2, min(_log(rng, 8, 16384), 2 ** 29 // page))
    return dict(op="compact", dtype=dt, NB=nb, live=rng.randint(0, 100), Hkv=H, D=D, bs=bs)


# --------------------------------------------------------------------------------------------
# Inputs.

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _evenly(lo, hi, n, gen):
    """n lengths spread evenly over [lo, hi], in an order drawn from the generator."""
    v = torch.tensor([hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)])
    return v[torch.randperm(n, generator=gen)].to(torch.int32)


def _state(dev, score, **parts):
    """The integers that a pass changes, in one buffer with a copy of what they were: one copy
    brings them back before the next pass.  Returns (buffer, copy, name -> view)."""
    parts = {k: v.to(torch.int32).reshape(v.shape) for k, v in parts.items()}
    flat = torch.cat([v.reshape(-1) for v in parts.values()] + [score.reshape(-1).view(torch.int32)]).to(dev)
    views, at = {}, 0
    for k, v in parts.items():
        views[k] = flat[at:at + v.numel()].view(v.shape)
        at += v.numel()
    views["score"] = flat[at:].view(torch.float32).view(score.shape)
    return flat, flat.clone(), views


def _rows(gen, dev, dt, *shape):
    """N(0,1) rows whose heads differ in size, as keys and values of trained models do."""
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16 if dt is torch.bfloat16 else torch.float32)
    size = torch.exp2(torch.rand((shape[-2], 1), generator=gen, device=dev) * 4 - 2)
    return (x * size).to(dt)


def _pages8(gen, dev, H, NB, bs, D):
    """A pool of e4m3 numbers and their scales, quantised page by page."""
    x = torch.randn((H, NB, bs, D), generator=gen, device=dev, dtype=torch.bfloat16)
    x *= torch.exp2(torch.rand((H, 1, 1, 1), generator=gen, device=dev) * 4 - 2).to(torch.bfloat16)
    s = _scale_for(x.abs().amax(dim=(2, 3)).float())
    return (x / s.to(torch.bfloat16)[:, :, None, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    dev = torch.device("cuda")
    cpu = torch.Generator().manual_seed(int(seed) * 7 + 1)
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    op, D = case["op"], case["D"]
    st = {"case": case}
    if op == "norm":
        dt, T = _TYPES[case["dtype"]], case["T"]
        st["q"], st["k"] = _rows(gen, dev, dt, T, case["Hq"], D), _rows(gen, dev, dt, T, case["Hkv"], D)
        st["wq"], st["wk"] = ((1 + 0.2 * torch.randn(D, generator=gen, device=dev)).to(dt) for _ in range(2))
        st["cos_sin"] = st["pos"] = None
        if case["rot"]:
            half = case["rot"] // 2
            i = torch.arange(half, dtype=torch.float64, device=dev)
            a = torch.arange(case["n_pos"], dtype=torch.float64, device=dev)[:, None] * 10000.0 ** (-i / half)
            st["cos_sin"] = torch.stack([a.cos(), a.sin()], dim=1).float()
            # a prompt's tokens in order; the tokens of a decode step anywhere
            p = torch.arange(T) % case["n_pos"] if T > 256 else torch.randint(0, case["n_pos"], (T,), generator=cpu)
            st["pos"] = p.to(torch.int32).to(dev)
    elif op == "append":
        dt, B, H, bs = _TYPES[case["dtype"]], case["B"], case["Hkv"], case["bs"]
        lens, new = _evenly(case["lo"], case["hi"], B, cpu), _evenly(case["new_lo"], case["new_hi"], B, cpu)
        nb, mb = (lens + bs - 1) // bs, int(((lens + new + bs - 1) // bs).max())
        NB = int(((lens + new + bs - 1) // bs).sum()) + 3
        perm, used = torch.randperm(NB, generator=cpu), int(nb.sum())
        st["n"] = int(new.sum())
        st["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).to(torch.int32).to(dev)
        st["kn"], st["vn"] = _rows(gen, dev, dt, st["n"], H, D), _rows(gen, dev, dt, st["n"], H, D)
        st["k"], st["ks"] = _pages8(gen, dev, H, NB, bs, D)
        st["v"], st["vs"] = _pages8(gen, dev, H, NB, bs, D)
        ids = torch.zeros(NB, dtype=torch.int32)
        ids[:NB - used] = perm[used:]
        st["flat"], st["before"], st["s"] = _state(
            dev, torch.zeros((B, mb)), table=_table(nb, mb, perm[:used]), len=lens, n_blocks=nb, ids=ids,
            top=torch.tensor([NB - used]))
    elif op == "decode":
        B, H, bs, Hq = case["B"], case["Hkv"], case["bs"], case["Hq"]
        lens = _evenly(case["lo"], case["hi"], B, cpu)
        nb = (lens + bs - 1) // bs
        mb, NB = max(1, int(nb.max())), int(nb.sum()) + 5
        st["scale"] = 1.0 / math.sqrt(D)
        st["q"] = _rows(gen, dev, _TYPES[case["dtype"]], B, Hq, D)
        st["k"], st["ks"] = _pages8(gen, dev, H, NB, bs, D)
        st["v"], st["vs"] = _pages8(gen, dev, H, NB, bs, D)
        # attention sinks: the first page of every sequence weighs more
        table = _table(nb, mb, torch.randperm(NB, generator=cpu)[:int(nb.sum())])
        st["ks"][:, table[:, 0].long().to(dev)] *= 2.0
        _, _, st["s"] = _state(dev, torch.zeros((B, mb)), table=table, len=lens, n_blocks=nb)
    elif op == "reorder":
        B, g, bs = case["B"], case["group"], case["bs"]
        lens = _evenly(case["lo"], case["hi"], B // g, cpu).repeat_interleave(g)   # beams are equally long
        nb = (lens + bs - 1) // bs
        mb = max(1, int(nb.max()))
        shared = (lens // bs) * 3 // 4               # the pages of the prompt, held by all beams
        owns = torch.where(torch.arange(B) % g == 0, nb, nb - shared)
        table, shares, at = torch.zeros((B, mb), dtype=torch.int32), [], int(owns.sum())
        NB = at + B + 2
        perm = torch.randperm(NB, generator=cpu).to(torch.int32)
        shares, at = torch.zeros(NB, dtype=torch.int32), 0
        for b in range(B):
            n, s = int(nb[b]), int(shared[b])
            if b % g:
                table[b, :s] = table[b - b % g, :s]
                shares[table[b, :s].long()] += 1
            else:
                s = 0
            table[b, s:n] = perm[at:at + n - s]
            at += n - s
        ids = torch.zeros(NB, dtype=torch.int32)
        ids[:NB - at] = perm[at:]
        # every beam goes on from one of its prompt's; about one prompt in eight is done
        parent = torch.arange(B) // g * g + torch.randint(0, g, (B,), generator=cpu)
        done = torch.rand(B // g, generator=cpu) < (0.125 if g > 1 else 0.5)
        st["parent"] = torch.where(done.repeat_interleave(g), torch.tensor(-1), parent).to(torch.int32).to(dev)
        _pool(st, case, gen, dev, NB)
        st["flat"], st["before"], st["s"] = _state(
            dev, torch.rand((B, mb), generator=cpu), table=table, len=lens, n_blocks=nb, shares=shares, ids=ids,
            top=torch.tensor([NB - at]))
    else:
        NB, bs = case["NB"], case["bs"]
        live = NB * case["live"] // 100
        perm = torch.randperm(NB, generator=cpu).to(torch.int32)
        B = max(1, min(16, live))
        nb = torch.tensor([live * (b + 1) // B - live * b // B for b in range(B)], dtype=torch.int32)
        mb = max(1, int(nb.max()))
        ids = torch.zeros(NB, dtype=torch.int32)
        ids[:NB - live] = perm[live:]
        _pool(st, case, gen, dev, NB)
        st["flat"], st["before"], st["s"] = _state(
            dev, torch.zeros((B, mb)), table=_table(nb, mb, perm[:live]), len=nb * bs, n_blocks=nb,
            shares=torch.zeros(NB), ids=ids, top=torch.tensor([NB - live]))
    if own:
        _plan(st)
    return st


def _table(nb, mb, ids):
    """[B, mb] page table: sequence b's nb[b] entries in order from ids, the others 0."""
    t = torch.zeros((len(nb), mb), dtype=torch.int32)
    t[torch.arange(mb) < nb[:, None]] = ids.to(torch.int32)
    return t


def _pool(st, case, gen, dev, NB):
    H, bs, D = case["Hkv"], case["bs"], case["D"]
    if case["dtype"] == "e4m3":
        st["k"], st["ks"] = _pages8(gen, dev, H, NB, bs, D)
        st["v"], st["vs"] = _pages8(gen, dev, H, NB, bs, D)
    else:
        for x in ("k", "v"):
            st[x] = torch.randn((H, NB, bs, D), generator=gen, device=dev, dtype=_TYPES[case["dtype"]])


def _plan(st):
    """What a program keeps between calls: the library's descriptors and workspace."""
    from kv_cache_compression_kvc_gb300 import kvc
    c, s, dev = st["case"], st.get("s"), st.get("k").device
    if c["op"] == "norm":
        return
    st["pool"] = kvc.block_pool_q8_view(st["k"], st["v"], st["ks"], st["vs"]) if "ks" in st else \
        kvc.block_pool_view(st["k"], st["v"])
    st["pt"] = kvc.page_table_view(s["table"], s["n_blocks"], s["len"], s["score"])
    B, mb = s["table"].shape
    if c["op"] == "decode":
        st["ws"] = kvc.decode_q8_workspace(c["B"], c["Hq"], c["Hkv"], c["D"], st["q"].dtype, dev)
        return
    st["free"] = kvc.free_pool_view(s["ids"], s["top"])
    if c["op"] == "append":
        st["ws"] = kvc.append_q8_workspace(B, st["n"], c["bs"], dev)
    else:
        st["ws"] = kvc.pages_workspace(B, mb, st["k"].shape[1], dev)


# --------------------------------------------------------------------------------------------
# One pass.


def run(st):
    return {"norm": _run_norm, "append": _run_append, "decode": _run_decode, "reorder": _run_reorder,
            "compact": _run_compact}[st["case"]["op"]](st)


_EPS = 1e-6


def _run_norm(st):
    if own:
        from kv_cache_compression_kvc_gb300 import kvc
        return kvc.kvc_qk_norm_rope(st["q"], st["k"], w_q=st["wq"], w_k=st["wk"], eps=_EPS, cos_sin=st["cos_sin"], pos=st["pos"])
    return _plain_norm(st, st["q"], st["wq"]), _plain_norm(st, st["k"], st["wk"])


def _plain_norm(st, x, w):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(dim=-1, keepdim=True) + _EPS) * w.float()
    rot = st["case"]["rot"]
    if rot:
        c = st["cos_sin"][st["pos"].long()][:, None]                      # [T, 1, 2, rot/2]
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        y = torch.cat([a * c[:, :, 0] - b * c[:, :, 1], b * c[:, :, 0] + a * c[:, :, 1], y[..., rot:]], dim=-1)
    return y.to(x.dtype)


def _scale_for(amax):
    """The smallest power of two s with amax / s <= 448, e4m3's largest number: 448 is 1.75 * 2^8."""
    bits = amax.view(torch.int32)
    e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    return ((e.clamp(-120, 119) + 127) << 23).view(torch.float32)


def _run_append(st):
    c, s = st["case"], st["s"]
    st["flat"].copy_(st["before"])                  # the program's tables before this step
    if own:
        from kv_cache_compression_kvc_gb300 import kvc
        kvc.kvc_paged_append_q8(st["pool"], st["pt"], st["free"], st["kn"], st["vn"], cu=st["cu"], ws=st["ws"])
    else:
        B, bs, dev = c["B"], c["bs"], st["k"].device
        mb = s["table"].shape[1]
        new = st["cu"][1:] - st["cu"][:-1]
        end = (s["len"] + new + bs - 1) // bs
        need = end - s["n_blocks"]
        before = need.cumsum(0) - need
        i = torch.arange(mb, device=dev)
        opens = (i >= s["n_blocks"][:, None]) & (i < end[:, None])
        at = s["top"] - 1 - (before[:, None] + i - s["n_blocks"][:, None])
        s["table"].copy_(torch.where(opens, s["ids"][at.clamp(0, s["ids"].numel() - 1).long()], s["table"]))
        s["score"].masked_fill_(opens, 0.0)
        # the sequence, page and row of every new token
        tok = torch.arange(st["n"], device=dev)
        b = torch.searchsorted(st["cu"][1:].contiguous(), tok.to(torch.int32), right=True)
        where = s["len"][b] + tok - st["cu"][b]
        page = s["table"][b, where // bs].long()
        part = s["table"].gather(1, (s["len"] // bs).clamp(max=mb - 1).long()[:, None])[:, 0].long()
        held = s["len"] % bs                        # rows that those pages hold already
        for new_rows, pool, scale in ((st["kn"], st["k"], st["ks"]), (st["vn"], st["v"], st["vs"])):
            _plain_quantise(new_rows, pool, scale, page, where % bs, part, held)
        s["top"].sub_(need.sum())
        s["len"].add_(new)
        s["n_blocks"].copy_(end)
    return st["k"], st["v"], st["ks"], st["vs"], s["table"], s["n_blocks"], s["len"], s["score"], s["top"]


def _plain_quantise(rows, pool, scale, page, row, part, held):
    x = rows.float()                                                      # [n, H, D]
    H, NB = scale.shape
    amax = torch.zeros((NB, H), device=x.device).index_reduce_(0, page, x.abs().amax(dim=2), "amax")
    touched = torch.zeros(NB, dtype=torch.bool, device=x.device).index_fill_(0, page, True)
    old = torch.zeros_like(scale).index_copy_(1, part, torch.where(held > 0, scale[:, part], torch.zeros((), device=x.device)))
    now = torch.where(touched, torch.maximum(old, _scale_for(amax.T.contiguous())), scale)
    # the rows that a partly filled page held go over to its new scale
    r8 = pool.view(torch.uint8)
    p8 = r8[:, part].view(torch.float8_e4m3fn).float() * (scale[:, part] / now[:, part])[:, :, None, None]
    keep = (torch.arange(pool.shape[2], device=x.device) < held[:, None])[None, :, :, None]
    r8[:, part] = torch.where(keep, p8.to(torch.float8_e4m3fn).view(torch.uint8), r8[:, part])
    y = x / now[:, page].T[:, :, None]
    r8[:, page, row] = y.to(torch.float8_e4m3fn).view(torch.uint8).transpose(0, 1)
    scale.copy_(now)


def _run_decode(st):
    q, s = st["q"], st["s"]
    if own:
        from kv_cache_compression_kvc_gb300 import kvc
        lse = torch.empty(q.shape[:2], device=q.device)
        out = kvc.kvc_decode_attn_paged_q8(q, st["pool"], st["pt"], scale=st["scale"], lse=lse, ws=st["ws"])
        return out, lse
    B, Hq, D = q.shape
    k, v = _plain_pages(st["k"], st["ks"], s["table"]), _plain_pages(st["v"], st["vs"], s["table"])
    H, S = k.shape[1], k.shape[2]
    x = (q.float().view(B, H, Hq // H, D) @ k.transpose(2, 3)) * st["scale"]
    x = x.masked_fill(~(torch.arange(S, device=q.device) < s["len"][:, None])[:, None, None], float("-inf"))
    m = x.amax(dim=3, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    z = p.sum(dim=3, keepdim=True)
    v = torch.where((torch.arange(S, device=q.device) < s["len"][:, None])[:, None, :, None], v, torch.zeros((), device=q.device))
    o = (p @ v) / torch.where(z == 0, torch.ones_like(z), z)
    return o.view(B, Hq, D).to(q.dtype), (m + torch.log(z))[..., 0].view(B, Hq)


def _plain_pages(pool, scale, table):
    """[H, NB, bs, D] e4m3 with scales [H, NB], through table [B, mb] -> fp32 [B, H, mb * bs, D]."""
    t = table.long()
    x = pool.view(torch.uint8)[:, t].view(torch.float8_e4m3fn).float() * scale[:, t][..., None, None]
    return x.permute(1, 0, 2, 3, 4).flatten(2, 3)


def _run_reorder(st):
    c, s = st["case"], st["s"]
    st["flat"].copy_(st["before"])
    if own:
        from kv_cache_compression_kvc_gb300 import kvc
        kvc.kvc_pages_reorder(st["pool"], st["pt"], st["free"], s["shares"], st["parent"], ws=st["ws"])
    else:
        B, bs, dev, par = c["B"], c["bs"], st["k"].device, st["parent"]
        mb, NB = s["table"].shape[1], st["k"].shape[1]
        me, i = torch.arange(B, device=dev), torch.arange(mb, device=dev)
        has, up = par >= 0, par.clamp(min=0).long()
        kids = torch.zeros(B, dtype=torch.int32, device=dev).index_add_(0, up, has.to(torch.int32))
        # a partly filled page stays with the sequence itself, else with its first child
        first = torch.full((B,), B, device=dev).scatter_reduce_(0, up, torch.where(has, me, torch.tensor(B, device=dev)), "amin")
        first = torch.where(par == me, me, first)
        held = s["len"] % bs
        last = (held > 0)[:, None] & (i == s["n_blocks"][:, None] - 1)
        change = torch.where((i < s["n_blocks"][:, None]) & ~(last & (kids > 0)[:, None]), kids[:, None] - 1, torch.zeros((), dtype=torch.int32, device=dev))
        shares = s["shares"].index_add(0, s["table"].reshape(-1).long(), change.reshape(-1))
        gone = shares < 0
        freed = torch.zeros(NB + 1, dtype=torch.int32, device=dev)
        freed.scatter_(0, torch.where(gone, gone.cumsum(0) - 1, NB), torch.arange(NB, dtype=torch.int32, device=dev))
        copies = has & (held[up] > 0) & (first[up] != me)
        rank, slot, n_gone = copies.cumsum(0) - 1, torch.arange(NB, device=dev), gone.sum()
        at = s["top"] + n_gone - 1 - rank
        take = torch.where(at >= s["top"], freed[(at - s["top"]).clamp(0, NB)], s["ids"][at.clamp(0, NB - 1)])
        top = s["top"] + n_gone - copies.sum()
        s["ids"].copy_(torch.where((slot >= s["top"]) & (slot < top), freed[(slot - s["top"]).clamp(0, NB)], s["ids"]))
        s["top"].copy_(top)
        s["shares"].copy_(torch.where(gone, torch.zeros_like(shares), shares))
        w = copies.nonzero()[:, 0]
        src, dst = s["table"][up[w], s["n_blocks"][up[w]] - 1].long(), take[w].long()
        keep = (torch.arange(bs, device=dev) < held[up[w]][:, None])[None, :, :, None]
        for x in ("k", "v"):
            pool = st[x].view(torch.uint8) if c["dtype"] == "e4m3" else st[x]
            pool[:, dst] = torch.where(keep, pool[:, src], pool[:, dst])
            if c["dtype"] == "e4m3":
                st[x + "s"][:, dst] = st[x + "s"][:, src]
        live = has[:, None] & (i < s["n_blocks"][up][:, None])
        table = torch.where(copies[:, None] & last[up], take[:, None].to(torch.int32), s["table"][up])
        s["table"].copy_(torch.where(live, table, s["table"]))
        s["score"].copy_(torch.where(live, s["score"][up], s["score"]))
        s["len"].copy_(torch.where(has, s["len"][up], 0))
        s["n_blocks"].copy_(torch.where(has, s["n_blocks"][up], 0))
    out = [st["k"], st["v"], s["table"], s["n_blocks"], s["len"], s["score"], s["shares"], s["ids"], s["top"]]
    return out + [st["ks"], st["vs"]] if "ks" in st else out


def _run_compact(st):
    c, s = st["case"], st["s"]
    st["flat"].copy_(st["before"])
    NB, dev = c["NB"], st["k"].device
    if own:
        from kv_cache_compression_kvc_gb300 import kvc
        remap = kvc.kvc_pages_compact(st["pool"], st["pt"], st["free"], shares=s["shares"], ws=st["ws"])
    else:
        slot = torch.arange(NB, device=dev, dtype=torch.int32)
        free = torch.zeros(NB + 1, dtype=torch.bool, device=dev)
        free.index_fill_(0, torch.where(slot < s["top"], s["ids"], NB).long(), True)
        free = free[:NB]
        n_live = NB - s["top"]
        moves, hole = ~free & (slot >= n_live), free & (slot < n_live)
        holes = torch.zeros(NB + 1, dtype=torch.int32, device=dev)
        holes.scatter_(0, torch.where(hole, hole.cumsum(0) - 1, NB), slot)
        remap = torch.where(moves, holes[(moves.cumsum(0) - 1).clamp(min=0)], torch.where(free, -1, slot))
        src = moves.nonzero()[:, 0]
        dst = remap[src].long()
        for x in ("k", "v"):
            pool = st[x].view(torch.uint8) if c["dtype"] == "e4m3" else st[x]
            pool[:, dst] = pool[:, src]
            if c["dtype"] == "e4m3":
                st[x + "s"][:, dst] = st[x + "s"][:, src]
        s["shares"][dst] = s["shares"][src]
        s["shares"][src] = 0
        valid = torch.arange(s["table"].shape[1], device=dev) < s["n_blocks"][:, None]
        s["table"].copy_(torch.where(valid, remap[s["table"].long()], s["table"]))
        s["ids"].copy_(torch.where(slot < s["top"], NB - 1 - slot, s["ids"]))
    out = [st["k"], st["v"], s["table"], s["shares"], s["ids"], s["top"], remap]
    return out + [st["ks"], st["vs"]] if "ks" in st else out


# --------------------------------------------------------------------------------------------
# The definitions in 64 bits.


def _power(e):
    """2^e in 64 bits, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """x (64 bits, at most 448 in size) to the nearest e4m3 number: 4 significant bits, steps of 2^-9 below 2^-6."""
    e = torch.frexp(x.abs().clamp(min=2.0 ** -6))[1]             # 2^(e - 1) <= |x| < 2^e
    step = _power(e - 4)
    return torch.round(x / step) * step


def exact(case, seed):
    op, D = case["op"], case["D"]
    if op in ("reorder", "compact"):
        return None                                # copies: nothing is computed
    st = prepare(case, seed)
    if op == "norm":
        out = []
        for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
            y = x.double()
            y = y / torch.sqrt((y * y).sum(dim=2, keepdim=True) / D + _EPS) * w.double()
            if case["rot"]:
                h = case["rot"] // 2
                cs = st["cos_sin"].double()[st["pos"].long()]
                z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.zeros((), dtype=torch.float64, device="cuda"))
                z = torch.complex(cs[:, 0], cs[:, 1])[:, None] * z
                r = torch.complex(y[..., :h].contiguous(), y[..., h:2 * h].contiguous()) * z
                y[..., :h], y[..., h:2 * h] = r.real, r.imag
            out.append(y)
        return tuple(out)
    s = st["s"]
    lens, H, bs = s["len"].tolist(), case["Hkv"], case["bs"]
    if op == "append":
        cu, top, table = st["cu"].tolist(), int(s["top"]), s["table"].tolist()
        ids, out = s["ids"].tolist(), []
        place = []                                 # (page, rows held, first new row, rows) in order
        for b, n in enumerate(lens):
            at, end = n, n + cu[b + 1] - cu[b]
            while at < end:
                if at % bs == 0:
                    top -= 1
                    table[b][at // bs] = ids[top]
                k = min(bs - at % bs, end - at)
                place.append((table[b][at // bs], at % bs, cu[b] + at - n, k))
                at += k
        if len(place) > 6000:
            return None
        for rows, pool, scale in ((st["kn"], st["k"], st["ks"]), (st["vn"], st["v"], st["vs"])):
            pool, scale = pool.double(), scale.double()
            for page, held, row, k in place:
                x = rows[row:row + k].double().transpose(0, 1)            # [H, k, D]
                big = x.abs().amax(dim=(1, 2)).clamp(min=2.0 ** -119)
                m, e = torch.frexp(big / 448.0)                           # m * 2^e, m in [1/2, 1)
                want = _power(e - (m == 0.5).to(e.dtype))
                if held:
                    was = scale[:, page].clone()
                    want = torch.maximum(want, was)
                    pool[:, page, :held] = _e4m3(pool[:, page, :held] * (was / want)[:, None, None])
                pool[:, page, held:held + k] = _e4m3(x / want[:, None, None])
                scale[:, page] = want
            out.append((pool, scale))
        return out[0][0], out[1][0], out[0][1], out[1][1], None, None, None, None, None
    B, Hq = case["B"], case["Hq"]
    G = Hq // H
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        pages = s["table"][b, : -(-n // bs)].long()
        for h in range(H):
            if n == 0:
                continue
            k, v = ((x[h].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double() * y[h, pages].double()[:, None, None]).flatten(0, 1)[:n]
                    for x, y in ((st["k"], st["ks"]), (st["v"], st["vs"])))
            x = st["q"][b, h * G:(h + 1) * G].double() @ k.T * st["scale"]
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, dim=1)
            out[b, h * G:(h + 1) * G] = torch.softmax(x, dim=1) @ v
    return out, lse


# --------------------------------------------------------------------------------------------
# What a pass cannot do without.


def _total(lo, hi, n):
    return hi if n == 1 else sum(lo + (hi - lo) * i // (n - 1) for i in range(n))


def work(case):
    op, D = case["op"], case["D"]
    es = {"bf16": 2, "fp32": 4, "e4m3": 1}[case["dtype"]]
    if op == "norm":
        n = case["T"] * (case["Hq"] + case["Hkv"]) * D
        # every row in and out, and the cosines and sines of every position once
        return {"bytes": 2 * n * es + min(case["T"], case["n_pos"]) * case["rot"] * 4, "flops": 8 * n}
    H, bs = case["Hkv"], case["bs"]
    if op == "append":
        n = 2 * _total(case["new_lo"], case["new_hi"], case["B"]) * H * D
        return {"bytes": n * (es + 1), "flops": 3 * n}
    if op == "decode":
        B, Hq = case["B"], case["Hq"]
        slots = _total(case["lo"], case["hi"], B) * H
        return {"bytes": 2 * slots * D + 2 * slots / bs * 4 + 2 * B * Hq * D * es + 4 * B * Hq,
                "flops": 4 * slots * (Hq // H) * D}
    if op == "reorder":
        # of g beams that pick a parent each, g (1 - 1/g)^g parents are picked by nobody, and as many
        # beams need a partly filled page of their own (half full on average, seven prompts in eight)
        B, g = case["B"], case["group"]
        n = 0.875 * B * (1 - 1 / g) ** g * H * D * bs / 2 * es * 2
        return {"bytes": 2 * n + 2 * 8 * _total(case["lo"], case["hi"], B) / bs + 16 * B, "flops": 0}
    # the live pages above the number of live pages are read once and written once
    a = case["live"] / 100
    return {"bytes": 2 * 2 * case["NB"] * a * (1 - a) * H * bs * D * es + 16 * case["NB"], "flops": 0}
