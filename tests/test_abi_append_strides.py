"""Appending to 8-bit pages: the stride of a single row or a single head means nothing, and may differ between keys and
values; every other one has to be the same.  On the CPU, with the library's call recorded instead of made."""
import pytest
import torch

from test_abi_pages_q8 import B, D, H, append_call, kvc  # noqa: F401


def sliced(n, heads, width):
    """[n, heads, D] out of rows of `width` heads."""
    return torch.zeros(n, width, D)[:, 1:1 + heads]


def test_one_row_beside_a_projection(kvc):  # noqa: F811
    append_call(kvc, k_new=torch.zeros(1, H, D), v_new=sliced(1, H, 9))
    append_call(kvc, k_new=sliced(1, H, 5), v_new=sliced(1, H, 9))
    odd = torch.zeros(1000).as_strided((1, H, D), (13, D, 1))
    append_call(kvc, k_new=odd, v_new=odd)
    append_call(kvc, k_new=torch.zeros(0, H, D), v_new=sliced(0, H, 9))
    assert len(kvc.stub_calls) == 4


def test_other_strides_are_refused(kvc):  # noqa: F811
    for k, v in ((torch.zeros(2, H, D), sliced(2, H, 9)), (torch.zeros(1, H, D), torch.zeros(1, H, 2 * D)[..., :D]),
                 (torch.zeros(1, H, D), torch.zeros(2, H, D)), (torch.zeros(1, H, D), torch.zeros(1, H + 1, D))):
        with pytest.raises(ValueError):
            append_call(kvc, k_new=k, v_new=v)
    assert not kvc.stub_calls
