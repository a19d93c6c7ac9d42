"""One token of one sequence: keys from the norms, contiguous, beside values that lie in the projection's output; and
one head, whose stride means nothing either."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,H,Hq", [(1, 2, 4), (1, 1, 3), (37, 1, 0)])
def test_normed_keys_beside_projected_values(dt, n, H, Hq):
    from kv_cache_compression_kvc_gb300 import kvc
    D, bs, NB = 64, 16, 4
    g = torch.Generator(device=DEV).manual_seed(1)
    k = torch.randn((n, H, D), generator=g, device=DEV).to(dt)
    qkv = torch.randn((n, Hq + 2 * H, D), generator=g, device=DEV).to(dt)
    v = qkv[:, Hq + H:] if n == 1 else qkv[:, 0].clone()[:, None].as_strided((n, 1, D), (D, 5 * D, 1))
    runs = []
    for values in (v, v.clone(memory_format=torch.contiguous_format)):
        pools = [torch.zeros((H, NB, bs, D), dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = [torch.zeros((H, NB), device=DEV) for _ in range(2)]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        table, nb, lens = i32([[0] * 4]), i32([0]), i32([0])
        pt = kvc.page_table_view(table, nb, lens, torch.zeros((1, 4), device=DEV))
        free = kvc.free_pool_view(torch.arange(NB, dtype=torch.int32, device=DEV), i32([NB]))
        pool = kvc.block_pool_q8_view(*pools, *scales)
        for _ in range(2):
            kvc.kvc_paged_append_q8(pool, pt, free, k[:24], values[:24], cu=i32([0, min(n, 24)]))
        assert kvc.kvc_device_status() == 0 and int(lens) == 2 * min(n, 24)
        runs.append(pools + scales)
    assert all(torch.equal(x, y) for x, y in zip(*runs))
