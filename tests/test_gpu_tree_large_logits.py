"""GPU: logits of any finite size.  Keys of equal components, powers of two and 1.375 times those, make the
logits exact (the second kind not their products with the scale in base-2 units), the largest one
shared by every third slot or so and the others far below it: the output is the mean of the values
there, however large or how far below zero the logits lie."""
import pytest
import torch

from gpu_helpers import cuda_or_skip, lib
from tree_ref import compare, randn

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]


def keys(rows, sign, base, exponent, seed, dev, dtype):
    """rows x 1 factors of the largest logit: 1 for about a third of them (the first among them), else
    so much less that their weight is 0."""
    gen = torch.Generator().manual_seed(seed)
    best = torch.rand(rows, generator=gen) < 0.35
    best[..., 0] = True
    low = 0.5 if sign > 0 else 2.0
    f = torch.where(best, torch.tensor(1.0), torch.tensor(low)) * sign * base * 2.0 ** exponent
    return f.to(dev, dtype), best.to(dev)


def check(out, lse, values, best, logit, dtype):
    """values [B, H, n, Dv], best [B, H, n], out [B, T, H, G, Dv].  The weights are 0 and one number near 1:
    what is left are the sums of n terms in fp32 (2^-23 each), the exponential and the quotient, the
    rounding of the weights (bf16 only, 2^-8) and that of the output (2^-8, fp32 2^-24)."""
    w = best.double()
    n = values.shape[2]
    count = w.sum(2)
    mean = torch.einsum("bhn,bhnd->bhd", w, values.double()) / count[..., None]
    size = torch.einsum("bhn,bhnd->bhd", w, values.double().abs()) / count[..., None]
    eps, weights = (2.0 ** -8, 2.0 ** -8) if dtype == torch.bfloat16 else (2.0 ** -24, 0.0)
    rel = (2 * n + 8) * 2.0 ** -23 + weights
    tol = rel * size + eps * (mean.abs() + rel * size) + 1e-30
    B, T, H, G, D = out.shape
    want, tol = (x[:, None, :, None].expand(B, T, H, G, D) for x in (mean, tol))
    compare(out, want, tol, "out")
    # the largest logit to its last places (two rounded products and a sum), log(count) in fp32
    z = (logit + torch.log(count))[:, None, :, None].expand(B, T, H, G)
    compare(lse, z, 2.0 ** -21 * z.abs() + 2.0 ** -18, "lse")


LEVELS = [(1, 10), (-1, 10), (1, 26), (-1, 33), (1, 34), (1, 60), (-1, 60), (1, 112), (-1, 112)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("base", [1.0, 1.375])
@pytest.mark.parametrize("sign,level", LEVELS)
@pytest.mark.parametrize("H,G,D,T,n", [(2, 2, 64, 4, 300), (1, 4, 128, 64, 700), (2, 6, 256, 11, 200),
                                       (1, 1, 128, 1, 20000), (1, 4, 128, 40, 9000)])
def test_tree(dtype, base, sign, level, H, G, D, T, n):
    dev = cuda_or_skip()
    kvc = lib()
    B = 2
    half = level // 2
    q = torch.full((B, T, H * G, D), 2.0 ** half, dtype=dtype, device=dev)
    f, best = keys((B, H, n), sign, base, level - half, 1, dev, dtype)
    k = f[..., None].expand(B, H, n, D).contiguous()
    v = randn((B, H, n, D), 2, dev, dtype)
    # a drafted token has the largest logit too; the mask shows it to every token
    kd = torch.full((B, T, H, D), 2.0 * sign * base * 2.0 ** (level - half) if sign < 0 else 0.0, dtype=dtype, device=dev)
    kd[:, 0] = sign * base * 2.0 ** (level - half)
    vd = randn((B, T, H, D), 3, dev, dtype)
    mask = torch.full((B, T), 1, dtype=torch.int64, device=dev) | (1 << torch.arange(T, device=dev))
    lse = torch.empty(q.shape[:3], device=dev)
    out = kvc.kvc_decode_attn_tree(q, kvc.cache_view(k, v), kvc.make_draft(kd, vd, mask=mask), scale=1.0,
                                   n_valid=n, lse=lse)
    assert kvc.kvc_device_status() == 0
    values = torch.cat([v, vd[:, :1].transpose(1, 2)], 2)
    best = torch.cat([best, torch.ones_like(best[..., :1])], 2)
    check(out.view(B, T, H, G, D), lse.view(B, T, H, G), values, best, sign * base * 2.0 ** level * D, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,G,T,n", [(2, 2, 4, 300), (1, 4, 40, 9000)])
def test_tree_at_the_lowest(dtype, H, G, T, n):
    """Logits that are among the lowest finite numbers in base-2 units; the others are -inf."""
    test_tree(dtype, 1.25, -1, 121, H, G, 64, T, n)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("base", [1.0, 1.375])
@pytest.mark.parametrize("sign,level", LEVELS)
@pytest.mark.parametrize("Hq,R,E,T,n", [(16, 512, 64, 1, 3000), (32, 256, 64, 4, 400)])
def test_latent(dtype, base, sign, level, Hq, R, E, T, n):
    """The keys' size stands in the rope part, the values in the latent one, where the query is 0."""
    dev = cuda_or_skip()
    kvc = lib()
    B = 2
    half = level // 2
    q = torch.zeros((B, T, Hq, R + E), dtype=dtype, device=dev)
    q[..., R:] = 2.0 ** half
    c = randn((B, n, R + E), 2, dev, dtype)
    f, best = keys((B, 1, n), sign, base, level - half, 1, dev, dtype)
    c[..., R:] = f[:, 0, :, None]
    cd = randn((B, T, R + E), 3, dev, dtype)
    cd[..., R:] = 2.0 * sign * base * 2.0 ** (level - half) if sign < 0 else 0.0
    lse = torch.empty(q.shape[:3], device=dev)
    out = kvc.kvc_decode_attn_latent(q, kvc.latent_cache_view(c, R), kvc.make_draft(cd), scale=1.0, n_valid=n, lse=lse)
    assert kvc.kvc_device_status() == 0
    check(out[:, :, None], lse[:, :, None], c[:, None, :, :R], best, sign * base * 2.0 ** level * E, dtype)
