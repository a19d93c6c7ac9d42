"""Plain 64-bit definitions of the draft-tree and latent operators, and the tolerances of their
tests (imported by tests only)."""
import torch

from kv_cache_compression_kvc_gb300 import inputs as I

SENTINEL = 123.0


def tree_masks(B, T, seed):
    """Ancestor bits of random trees: int64 [B, T] (the bits of a uint64)."""
    gen = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(B):
        words = []
        for t in range(T):
            parent = int(torch.randint(0, t + 1, (1,), generator=gen)) - 1
            words.append((words[parent] if parent >= 0 else 0) | (1 << t))
        out.append([w - (1 << 64) if w >> 63 else w for w in words])
    return torch.tensor(out, dtype=torch.int64)


def chain_masks(B, T):
    words = [(2 << t) - 1 for t in range(T)]
    return torch.tensor([[w - (1 << 64) if w >> 63 else w for w in words]] * B, dtype=torch.int64)


def attend(q, keys, values, kd, vd, mask, scale):
    """One (sequence, KV head): q [T, G, Dk]; keys/values the visible slots [n, .]; kd/vd the
    drafted rows [T, .] or None; mask [T] words.  Returns out, lse, and the quantities the error
    bounds need: sum p |v| and the largest scale * sum |q_i k_i| of each row."""
    q = q.double()
    n = keys.shape[0]
    if kd is not None:
        keys, values = torch.cat([keys, kd]), torch.cat([values, vd])
    keys, values = keys.double(), values.double()
    T = q.shape[0]
    s = torch.einsum("tgd,jd->tgj", q, keys) * scale
    mag = abs(scale) * torch.einsum("tgd,jd->tgj", q.abs(), keys.abs().nan_to_num(0, 0, 0))
    live = torch.ones(T, keys.shape[0], dtype=torch.bool, device=q.device)
    if kd is not None:
        for t in range(T):
            w = int(mask[t])
            for i in range(kd.shape[0]):
                live[t, n + i] = bool((w >> i) & 1)
    live = live[:, None].expand_as(s)
    s = torch.where(live, s, torch.full_like(s, float("-inf")))
    mag = torch.where(live, mag, torch.zeros_like(mag))
    if s.shape[2] == 0:
        z = torch.zeros(q.shape[:2] + (values.shape[1],), dtype=torch.float64, device=q.device)
        none = torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device=q.device)
        return z, none, z, torch.zeros_like(none)
    lse = torch.logsumexp(s, dim=2)
    p = torch.exp(s - torch.where(lse == float("-inf"), torch.zeros_like(lse), lse)[..., None])
    # a masked row contributes nothing whatever it holds
    out = torch.zeros(q.shape[:2] + (values.shape[1],), dtype=torch.float64, device=q.device)
    finite = torch.where(torch.isfinite(values), values, torch.zeros_like(values))
    out = torch.einsum("tgj,jd->tgd", p, finite)
    pv = torch.einsum("tgj,jd->tgd", p, finite.abs())
    for j in (~torch.isfinite(values).all(dim=1)).nonzero().flatten().tolist():
        bad = torch.where(torch.isfinite(values[j]), torch.zeros_like(values[j]), values[j])
        out = out + torch.where(live[:, :, j, None], bad, torch.zeros_like(bad))
    return out, lse, pv, mag.amax(dim=2)


def tolerance(dtype, width, n, pv, mag, out, lse):
    """Bounds on the errors of out and lse.

    Logits: a dot product of `width` terms accumulated in fp32 is off by at most width * 2^-23 of
    the sum of its terms' magnitudes (2^-24 a rounding to nearest, 2^-23 where the matrix unit
    truncates), in all ds = width * 2^-23 * mag.  A weight exp(s - lse) moves by at most 2 ds of itself
    (numerator and denominator), the base-2 exponential and the rescalings add 2^-20, the sums over
    n slots n * 2^-23 of the summed magnitudes; all these multiply sum p |v|.  With bf16 the
    weights are rounded (2^-8 of sum p |v|) and the output too (2^-8 of itself; fp32 2^-24).
    """
    ds = width * 2.0 ** -23 * mag
    rel = 2 * ds[..., None] + 2.0 ** -20 + 2 * n * 2.0 ** -23
    if dtype == torch.bfloat16:
        t_out = (rel + 2.0 ** -8) * pv + 2.0 ** -8 * (out.abs() + (rel + 2.0 ** -8) * pv)
    else:
        t_out = rel * pv + 2.0 ** -23 * out.abs()
    t_lse = ds + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -22 * lse.abs()
    return t_out + 1e-30, t_lse


def compare(got, ref, tol, what):
    got = got.double()
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    fin = torch.isfinite(ref)
    assert bool((same | fin).all()), f"{what}: infinities or NaN differ"
    err = torch.where(fin & ~same, (got - ref).abs(), torch.zeros_like(ref))
    over = ~(err <= torch.where(fin, tol, torch.ones_like(tol)))
    assert not bool(over.any()), (f"{what}: {int(over.sum())} of {over.numel()} beyond the bound; worst "
                                  f"{float((err - tol)[over].max()):.3g} over, error {float(err.max()):.3g}")


def check(out, lse, dtype, b_rows, what=""):
    """b_rows: iterable of (index into [B, T', heads], out, lse, pv, mag, width, n)."""
    for at, o, z, pv, mag, width, n in b_rows:
        t_out, t_lse = tolerance(dtype, width, n, pv, mag, o, z)
        compare(out[at], o, t_out, f"{what} out {at}")
        if lse is not None:
            compare(lse[at], z, t_lse, f"{what} lse {at}")


def randn(shape, seed, dev, dtype):
    return I.randn(shape, seed, dev, dtype)
