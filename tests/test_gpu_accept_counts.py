"""GPU: a count of drafted tokens outside 0..n_draft is recorded and clamped by every call that reads
it (see kvc_draft in kvc.h)."""
import pytest
import torch

from gpu_helpers import cuda_or_skip, lib
from tree_ref import randn

pytestmark = pytest.mark.gpu
BAD_INDEX, BAD_LENGTH = 3, 5


@pytest.mark.parametrize("form", ["contiguous", "paged", "latent"])
@pytest.mark.parametrize("count,n,status,want", [
    ([5, 2, 0], [4, 2, 0], BAD_LENGTH, [4, 2, 0]),        # more than n_draft: all of them
    ([4, 2 ** 31 - 1, 4], [1, 4, 0], BAD_LENGTH, [1, 4, 0]),
    ([4, -1, 4], [4, 0, 3], BAD_LENGTH, [4, 0, 3]),       # less than none: none, as is accepted
    ([4, -2 ** 31, 4], [4, 1, 3], None, [4, 0, 3]),       # and an entry of the path outside it
    ([4, 0, 3], [4, 0, 3], 0, [4, 0, 3]),
])
def test_accept_records_a_count_out_of_range(form, count, n, status, want):
    dev = cuda_or_skip()
    kvc = lib()
    B, H, D, T, bs = 3, 2, 64, 4, 4
    path = torch.arange(T, dtype=torch.int32, device=dev).repeat(B, 1)
    n_accept = torch.tensor(n, dtype=torch.int32, device=dev)
    counts = torch.tensor(count, dtype=torch.int32, device=dev)
    if form == "latent":
        c, cd = torch.zeros((B, 9, 192), device=dev), randn((B, T, 192), 1, dev, torch.float32)
        ln = torch.zeros(B, dtype=torch.int32, device=dev)
        kvc.kvc_latent_accept(kvc.latent_cache_view(c, 128), ln, kvc.make_draft(cd, count=counts), path, n_accept)
        rows = (c != 0).any(dim=2).sum(dim=1).tolist()
    else:
        draft = kvc.make_draft(*(randn((B, T, H, D), s, dev, torch.float32) for s in (1, 2)), count=counts)
        if form == "contiguous":
            k, v = torch.zeros((B, H, 9, D), device=dev), torch.zeros((B, H, 9, D), device=dev)
            lens = torch.zeros((B, H), dtype=torch.int32, device=dev)
            kvc.kvc_tree_accept(kvc.cache_view(k, v), lens, draft, path, n_accept)
            assert torch.equal(lens[:, 0], lens[:, 1])
            ln, rows = lens[:, 0], (k[:, 0] != 0).any(dim=2).sum(dim=1).tolist()
        else:
            kp, vp = torch.zeros((H, 8, bs, D), device=dev), torch.zeros((H, 8, bs, D), device=dev)
            table = torch.zeros((B, 3), dtype=torch.int32, device=dev)
            ln, nb = (torch.zeros(B, dtype=torch.int32, device=dev) for _ in range(2))
            free = torch.arange(8, dtype=torch.int32, device=dev)
            top = torch.tensor([8], dtype=torch.int32, device=dev)
            got = kvc.kvc_tree_accept_paged(
                kvc.block_pool_view(kp, vp), kvc.page_table_view(table, nb, ln, torch.zeros((B, 3), device=dev)),
                kvc.free_pool_view(free, top), draft, path, n_accept)
            assert got.tolist() == want
            rows = [sum(int((kp[0, i] != 0).any(dim=1).sum()) for i in table[b, :int(nb[b])]) for b in range(B)]
    code = kvc.kvc_device_status()
    # two refusals at once: the codes keep whichever came first
    assert code in (BAD_INDEX, BAD_LENGTH) if status is None else code == status
    assert ln.tolist() == want and rows == want
