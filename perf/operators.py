"""Measured cases of the draft-tree and latent-cache operators.

Each case is one pass through one operator.  With ``own`` false the pass is made of elementary
torch operations in fp32; with ``own`` true it is the call a user of the library makes.
"""
import math

import torch

own = False

# --------------------------------------------------------------------------------------------
# Cases.  op: "tree" (attention of a tree of drafted tokens over a contiguous cache), "paged"
# (the same over page tables of bs-token blocks), "accept" (append an accepted path), "latent"
# (absorbed latent attention), "expand" (latent rows to per-head keys and values).
# Lengths run evenly from lo to hi over the (batch, head) rows, or over the sequences for the
# caches that share a length among heads.


def listed():
    return [
        # a short prompt of the small test workload, four drafted tokens: latency of one call
        dict(name="tree_small", op="tree", dtype="bf16", B=1, Hq=8, Hkv=2, D=64, T=4, lo=128, hi=128),
        # the small workload in fp32, per-head budgets that differ, an odd tree
        dict(name="tree_fp32", op="tree", dtype="fp32", B=4, Hq=8, Hkv=2, D=64, T=13, lo=100, hi=2048),
        # the SnapKV workload's compressed cache verifying 16 drafted tokens per sequence
        dict(name="tree_snapkv", op="tree", dtype="bf16", B=4, Hq=32, Hkv=8, D=128, T=16, lo=5243, hi=5243),
        # an uncompressed 128k-token cache and a full 64-token tree: the most work per call
        dict(name="tree_long", op="tree", dtype="bf16", B=2, Hq=32, Hkv=8, D=128, T=64, lo=131072, hi=131072),
        # pyramid budgets (four to one over the rows), d_head 256, groups of six, odd tree
        dict(name="tree_pyramid", op="tree", dtype="bf16", B=2, Hq=24, Hkv=4, D=256, T=11, lo=3277, hi=13107),
        # the block-eviction workload: 16 sequences of 26 blocks, one query head per KV head
        dict(name="paged_blocks", op="paged", dtype="bf16", B=16, Hq=32, Hkv=32, D=128, T=8, lo=801, hi=832, bs=32),
        # accepting four of eight drafted tokens in a small batch: latency
        dict(name="accept_small", op="accept", dtype="bf16", B=4, Hq=8, Hkv=8, D=128, T=8, lo=100, hi=1000),
        # accepting up to 64 drafted tokens in a large batch of full-width caches
        dict(name="accept_large", op="accept", dtype="bf16", B=64, Hq=32, Hkv=32, D=128, T=64, lo=0, hi=128),
        # plain single-token decode over one short latent cache, 16 heads: latency
        dict(name="latent_one", op="latent", dtype="bf16", B=1, Hq=16, R=512, E=64, T=1, lo=1000, hi=1000),
        # a ragged serving batch, 16 heads, two tokens per sequence: the cache's bytes count
        dict(name="latent_batch", op="latent", dtype="bf16", B=32, Hq=16, R=512, E=64, T=2, lo=1024, hi=8192),
        # 128 heads and four drafted tokens: 512 rows against every latent row, products count
        dict(name="latent_heads", op="latent", dtype="bf16", B=8, Hq=128, R=512, E=64, T=4, lo=4096, hi=8192),
        # expanding a 4096-token prompt's latent rows to 32 heads of keys and values
        dict(name="expand_prompt", op="expand", dtype="bf16", B=2, Hq=32, R=512, E=64, D=128, lo=4096, hi=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges; costs no more than the largest listed one."""
    op = rng.choice(["tree", "tree", "paged", "accept", "latent", "latent", "expand"])
    dt = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("tree", "paged"):
        D = rng.choice([64, 128, 256])
        G = rng.choice([1, 2, 4, 6, 8])
        c = dict(op=op, dtype=dt, B=_log(rng, 1, 32), Hkv=rng.choice([1, 2, 3, 4, 8, 16]), D=D,
                 T=_log(rng, 1, 64))
        c["Hq"] = c["Hkv"] * G
        hi = _log(rng, 8, 32768) if rng.random() < 0.85 else rng.randint(0, 3)
        rows = c["B"] * c["Hkv"]
        limit = 2 ** 26 if dt == "bf16" else 2 ** 23        # elements of keys
        hi = max(1, min(hi, limit // (rows * D)))
        if dt == "fp32":                                    # products on the plain pipes
            hi = max(1, min(hi, 2 ** 32 // (rows * D * c["T"] * G)))
        c["hi"], c["lo"] = hi, rng.randint(0, hi)
        if op == "paged":
            c["bs"] = rng.choice([16, 32, 64])
    elif op == "accept":
        H = rng.choice([1, 3, 8, 32])
        c = dict(op=op, dtype=dt, B=_log(rng, 1, 64), Hq=H, Hkv=H, D=rng.choice([64, 128, 256]),
                 T=_log(rng, 1, 64), lo=0, hi=rng.randint(0, 300))
    elif op == "latent":
        c = dict(op=op, dtype=dt, B=_log(rng, 1, 32), Hq=rng.choice([1, 8, 16, 24, 32, 64, 128]),
                 R=rng.choice([256, 512]), E=rng.choice([32, 64]), T=_log(rng, 1, 16))
        hi = _log(rng, 8, 16384) if rng.random() < 0.85 else rng.randint(0, 3)
        limit = 2 ** 27 if dt == "bf16" else 2 ** 23        # rows of products
        hi = max(1, min(hi, limit // (c["B"] * c["Hq"] * c["T"])))
        c["hi"], c["lo"] = hi, rng.randint(0, hi)
    else:
        D = rng.choice([128, 256])
        c = dict(op=op, dtype=dt, B=_log(rng, 1, 4), Hq=rng.choice([1, 5, 8, 16, 32]),
                 R=rng.choice([256, 512]), E=rng.choice([32, 64]), D=D)
        limit = 2 ** 18 if dt == "bf16" else 2 ** 14        # token heads
        hi = _log(rng, 8, 4096) if rng.random() < 0.85 else rng.randint(0, 3)
        hi = max(1, min(hi, limit * 128 // D // (c["B"] * c["Hq"])))
        c["hi"], c["lo"] = hi, rng.randint(0, hi)
    return c


# --------------------------------------------------------------------------------------------
# Inputs.

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _lengths(case, n, gen):
    """n lengths spread evenly over [lo, hi], in an order drawn from the generator."""
    lo, hi = case["lo"], case["hi"]
    if n == 1:
        v = torch.tensor([hi])
    else:
        v = torch.tensor([lo + (hi - lo) * i // (n - 1) for i in range(n)])
    return v[torch.randperm(n, generator=gen)].to(torch.int32)


def _tree_mask(B, T, gen):
    """Ancestor bits of a random tree per sequence: int64 [B, T], bit i of word t set where
    drafted token t sees token i (itself and its ancestors)."""
    masks = []
    for _ in range(B):
        pick = torch.rand(T, generator=gen).tolist()
        words = []
        for t in range(T):
            parent = int(pick[t] * (t + 1)) - 1             # -1: a child of the last cached token
            w = (words[parent] if parent >= 0 else 0) | (1 << t)
            words.append(w)
        masks.append([w - (1 << 64) if w >> 63 else w for w in words])
    return torch.tensor(masks, dtype=torch.int64)


def prepare(case, seed):
    dev = torch.device("cuda")
    cpu = torch.Generator().manual_seed(int(seed) * 7 + 1)
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]

    def randn(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * scale).to(dt)

    op, B, Hq = case["op"], case["B"], case["Hq"]
    st = {"case": case}
    hi = max(case["hi"], 1)
    if op in ("tree", "paged"):
        Hkv, D, T = case["Hkv"], case["D"], case["T"]
        st["scale"] = 1.0 / math.sqrt(D)
        st["q"] = randn(B, T, Hq, D)
        st["kd"], st["vd"] = randn(B, T, Hkv, D), randn(B, T, Hkv, D)
        st["mask"] = _tree_mask(B, T, cpu).to(dev)
        if op == "tree":
            st["k"], st["v"] = randn(B, Hkv, hi, D), randn(B, Hkv, hi, D)
            # attention sinks: the first four keys lean towards the mean query
            lean = st["q"].float().mean(dim=(1, 2))
            lean = lean / lean.norm(dim=-1, keepdim=True).clamp_min(1e-9)
            st["k"][:, :, :4] += (2.0 * math.sqrt(D) * lean).to(dt)[:, None, None]
            st["len"] = _lengths(case, B * Hkv, cpu).view(B, Hkv).to(dev)
        else:
            bs = case["bs"]
            mb = -(-hi // bs)
            n_pool = B * mb + 7
            st["k"], st["v"] = randn(Hkv, n_pool, bs, D), randn(Hkv, n_pool, bs, D)
            perm = torch.randperm(n_pool, generator=cpu)[: B * mb].view(B, mb)
            st["table"] = perm.to(torch.int32).to(dev)
            st["len"] = _lengths(case, B, cpu).to(dev)
            st["n_blocks"] = ((st["len"] + bs - 1) // bs).to(torch.int32)
            st["score"] = torch.zeros((B, mb), device=dev)
    elif op == "accept":
        Hkv, D, T = case["Hkv"], case["D"], case["T"]
        cap = hi + T
        st["k"], st["v"] = randn(B, Hkv, cap, D), randn(B, Hkv, cap, D)
        st["kd"], st["vd"] = randn(B, T, Hkv, D), randn(B, T, Hkv, D)
        st["len0"] = _lengths(case, B * Hkv, cpu).view(B, Hkv).to(dev)
        # accepted paths: ascending drafted tokens, about half of them
        keep = torch.rand((B, T), generator=cpu) < 0.5
        order = torch.argsort((~keep).to(torch.int8), dim=1, stable=True)
        st["n_accept"] = keep.sum(dim=1).to(torch.int32).to(dev)
        st["path"] = order.to(torch.int32).to(dev)
    elif op == "latent":
        R, E, T = case["R"], case["E"], case["T"]
        st["scale"] = 1.0 / math.sqrt(192.0)
        st["q"] = randn(B, T, Hq, R + E, scale=0.6)
        st["c"] = randn(B, hi, R + E)
        st["cd"] = randn(B, T, R + E)
        st["mask"] = _tree_mask(B, T, cpu).to(dev)
        st["len"] = _lengths(case, B, cpu).to(dev)
    else:
        R, E, D = case["R"], case["E"], case["D"]
        st["c"] = randn(B, hi, R + E)
        st["wk"] = randn(Hq, D - E, R, scale=1.0 / math.sqrt(R))
        st["wv"] = randn(Hq, D, R, scale=1.0 / math.sqrt(R))
        st["len"] = _lengths(case, B, cpu).to(dev)
        st["k"] = torch.zeros((B, Hq, hi, D), device=dev, dtype=dt)
        st["v"] = torch.zeros((B, Hq, hi, D), device=dev, dtype=dt)
    if own:
        _plan(st)
    return st


def _plan(st):
    """What a program keeps between calls: the library's workspace and descriptors."""
    from kv_cache_compression_kvc_gb300 import kvc
    c = st["case"]
    if c["op"] in ("tree", "paged"):
        st["draft"] = kvc.make_draft(st["kd"], st["vd"], mask=st["mask"])
        st["ws"] = kvc.tree_workspace(c["B"], c["Hq"], c["Hkv"], c["D"], c["T"], st["k"].dtype, st["k"].device)
        if c["op"] == "paged":
            st["pool"] = kvc.block_pool_view(st["k"], st["v"])
            st["pt"] = kvc.page_table_view(st["table"], st["n_blocks"], st["len"], st["score"])
        else:
            st["cache"] = kvc.cache_view(st["k"], st["v"])
    elif c["op"] == "accept":
        st["draft"] = kvc.make_draft(st["kd"], st["vd"])
        st["cache"] = kvc.cache_view(st["k"], st["v"])
    elif c["op"] == "latent":
        st["draft"] = kvc.make_draft(st["cd"], mask=st["mask"])
        st["cache"] = kvc.latent_cache_view(st["c"], c["R"])
        st["ws"] = kvc.latent_workspace(c["B"], c["Hq"], c["R"], c["E"], c["T"], st["c"].dtype, st["c"].device)
    else:
        st["cache"] = kvc.latent_cache_view(st["c"], c["R"])
        st["dst"] = kvc.cache_view(st["k"], st["v"])


# --------------------------------------------------------------------------------------------
# One pass.


def run(st):
    op = st["case"]["op"]
    if op == "accept":
        return _run_accept(st)
    if op == "expand":
        return _run_expand(st)
    return _run_attention(st)


def _run_attention(st):
    op = st["case"]["op"]
    if own:
        from kv_cache_compression_kvc_gb300 import kvc
        q = st["q"]
        lse = torch.empty(q.shape[:3], device=q.device)
        if op == "tree":
            out = kvc.kvc_decode_attn_tree(q, st["cache"], st["draft"], scale=st["scale"], len=st["len"], lse=lse, ws=st["ws"])
        elif op == "paged":
            out = kvc.kvc_decode_attn_tree_paged(q, st["pool"], st["pt"], st["draft"], scale=st["scale"], lse=lse, ws=st["ws"])
        else:
            out = kvc.kvc_decode_attn_latent(q, st["cache"], st["draft"], scale=st["scale"], len=st["len"], lse=lse, ws=st["ws"])
        return out, lse
    if op == "tree":
        k, v, kd, vd, lens = st["k"].float(), st["v"].float(), st["kd"].float(), st["vd"].float(), st["len"]
    elif op == "paged":
        k, v = _pages(st["k"], st["table"]).float(), _pages(st["v"], st["table"]).float()
        kd, vd = st["kd"].float(), st["vd"].float()
        lens = st["len"][:, None]
    else:
        R = st["case"]["R"]
        k = st["c"].float()[:, None]
        v = k[..., :R]
        kd = st["cd"].float()[:, :, None]
        vd = kd[..., :R]
        lens = st["len"][:, None]
    return _plain_attention(st["q"], k, v, kd, vd, st["mask"], lens, st["scale"])


def _pages(pool, table):
    """[Hkv, n_pool, bs, D] through table [B, mb] -> [B, Hkv, mb * bs, D]."""
    x = pool[:, table.long()]
    return x.permute(1, 0, 2, 3, 4).flatten(2, 3)


def _plain_attention(q, k, v, kd, vd, mask, lens, scale):
    """q [B, T, Hq, Dk]; k, v [B, Hkv, S, .]; kd, vd [B, T, Hkv, .]; lens broadcasts to [B, Hkv]."""
    B, T, Hq, Dk = q.shape
    Hkv, S = k.shape[1], k.shape[2]
    G = Hq // Hkv
    rows = q.float().view(B, T, Hkv, G, Dk).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, Dk)
    kd, vd = kd.transpose(1, 2), vd.transpose(1, 2)                       # [B, Hkv, T, .]
    s = torch.cat([rows @ k.transpose(2, 3), rows @ kd.transpose(2, 3)], dim=3) * scale
    slot = torch.arange(S, device=q.device)
    bit = (mask[:, :, None] >> torch.arange(T, device=q.device)) & 1      # [B, T, T]
    see_cache = (slot < lens[..., None]).expand(B, Hkv, S)[:, :, None].expand(B, Hkv, T * G, S)
    see_draft = (bit != 0).repeat_interleave(G, dim=1)[:, None].expand(B, Hkv, T * G, T)
    s = s.masked_fill(~torch.cat([see_cache, see_draft], dim=3), float("-inf"))
    m = s.amax(dim=3, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    z = p.sum(dim=3, keepdim=True)
    p = p / torch.where(z == 0, torch.ones_like(z), z)
    o = p[..., :S] @ v + p[..., S:] @ vd
    lse = (m + torch.log(z))[..., 0]
    o = o.view(B, Hkv, T, G, -1).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, -1)
    return o.to(q.dtype), lse.view(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq)


def _run_accept(st):
    lens = st["len0"].clone()                      # the program's lengths before this step
    if own:
        from kv_cache_compression_kvc_gb300 import kvc
        kvc.kvc_tree_accept(st["cache"], lens, st["draft"], st["path"], st["n_accept"])
        return st["k"], st["v"], lens
    k, v, path, n = st["k"], st["v"], st["path"].long(), st["n_accept"]
    B, T = path.shape
    H, D = k.shape[1], k.shape[3]
    i = torch.arange(T, device=k.device)
    slot = (lens[:, :, None] + i).long()                                  # [B, H, T]
    take = (i < n[:, None])[:, None, :, None].expand(B, H, T, D)
    at = slot[..., None].expand(B, H, T, D)
    src = path[:, None, :, None].expand(B, H, T, D)
    k.scatter_(2, at, torch.where(take, st["kd"].transpose(1, 2).gather(2, src), k.gather(2, at)))
    v.scatter_(2, at, torch.where(take, st["vd"].transpose(1, 2).gather(2, src), v.gather(2, at)))
    return k, v, lens + n[:, None]


def _run_expand(st):
    if own:
        from kv_cache_compression_kvc_gb300 import kvc
        kvc.kvc_latent_expand(st["cache"], st["wk"], st["wv"], st["dst"], len=st["len"])
        return st["k"], st["v"]
    c, R, E = st["c"].float(), st["case"]["R"], st["case"]["E"]
    H, S = st["wk"].shape[0], c.shape[1]
    lat = c[:, None, :, :R]
    k = torch.cat([lat @ st["wk"].float().transpose(1, 2), c[:, None, :, R:].expand(-1, H, -1, E)], dim=3)
    v = lat @ st["wv"].float().transpose(1, 2)
    live = (torch.arange(S, device=c.device) < st["len"][:, None])[:, None, :, None]
    st["k"].copy_(torch.where(live, k.to(st["k"].dtype), st["k"]))
    st["v"].copy_(torch.where(live, v.to(st["v"].dtype), st["v"]))
    return st["k"], st["v"]


# --------------------------------------------------------------------------------------------
# The definition in 64 bits, sequence by sequence and head by head.


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "accept":
        return None                                # copies: nothing is computed
    if op == "expand":
        R = case["R"]
        k, v = st["k"].double(), st["v"].double()
        for b, n in enumerate(st["len"].tolist()):
            x = st["c"][b, :n].double()
            for h in range(case["Hq"]):
                k[b, h, :n] = torch.cat([x[:, :R] @ st["wk"][h].double().T, x[:, R:]], dim=1)
                v[b, h, :n] = x[:, :R] @ st["wv"][h].double().T
        return k, v
    B, T, Hq = case["B"], case["T"], case["Hq"]
    width = case["R"] if op == "latent" else case["D"]
    heads = 1 if op == "latent" else case["Hkv"]
    out = torch.zeros((B, T, Hq, width), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    lens = st["len"].tolist()
    # blocked[b][t, i]: drafted token t does not see token i
    blocked = [torch.tensor([[not (w >> i) & 1 for i in range(T)] for w in words], device="cuda")
               for words in st["mask"].tolist()]
    G = Hq // heads
    for b in range(B):
        for h in range(heads):
            if op == "tree":
                n = lens[b][h]
                k, v = st["k"][b, h, :n], st["v"][b, h, :n]
            elif op == "paged":
                n = lens[b]
                blocks = st["table"][b, : -(-n // case["bs"])].long()
                k, v = st["k"][h, blocks].flatten(0, 1)[:n], st["v"][h, blocks].flatten(0, 1)[:n]
            else:
                n = lens[b]
                k = st["c"][b, :n]
                v = k[:, : case["R"]]
            if op == "latent":
                kd = st["cd"][b]
                vd = kd[:, : case["R"]]
            else:
                kd, vd = st["kd"][b, :, h], st["vd"][b, :, h]
            keys = torch.cat([k, kd]).double()
            values = torch.cat([v, vd]).double()
            rows = st["q"][b, :, h * G:(h + 1) * G].double()              # [T, G, Dk]
            s = torch.einsum("tgd,jd->tgj", rows, keys) * st["scale"]
            s[:, :, n:] = s[:, :, n:].masked_fill(blocked[b][:, None], -math.inf)
            lse[b, :, h * G:(h + 1) * G] = torch.logsumexp(s, dim=2)
            out[b, :, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", torch.softmax(s, dim=2), values)
    return out, lse


# --------------------------------------------------------------------------------------------
# What a pass cannot do without.


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op, B, Hq = case["op"], case["B"], case["Hq"]

    def total(n):                                  # sum of the n lengths
        if n == 1:
            return case["hi"]
        return sum(case["lo"] + (case["hi"] - case["lo"]) * i // (n - 1) for i in range(n))

    if op in ("tree", "paged"):
        Hkv, D, T = case["Hkv"], case["D"], case["T"]
        slots = total(B * Hkv) if op == "tree" else total(B) * Hkv
        rows = T * Hq // Hkv
        return {"bytes": 2 * (slots + B * T * Hkv) * D * es + 2 * B * T * Hq * D * es + 4 * B * T * Hq,
                "flops": 4 * (slots + B * Hkv * T / 2) * rows * D}
    if op == "accept":
        # about half of the drafted tokens: each row read once and written once, keys and values
        return {"bytes": 2 * 2 * B * case["T"] / 2 * case["Hkv"] * case["D"] * es, "flops": 0}
    R, E = case["R"], case["E"]
    if op == "latent":
        T = case["T"]
        slots = total(B)
        return {"bytes": (slots + B * T) * (R + E) * es + B * T * Hq * (2 * R + E) * es + 4 * B * T * Hq,
                "flops": 2 * (slots + B * T / 2) * T * Hq * (2 * R + E)}
    D, slots = case["D"], total(B)
    return {"bytes": slots * (R + E) * es + Hq * (2 * D - E) * R * es + 2 * slots * Hq * D * es,
            "flops": 2 * slots * R * Hq * (2 * D - E)}
