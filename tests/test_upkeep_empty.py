"""Steps that have nothing to keep: attn_tree_accept takes no drafts at all, as attn_decode_tree does."""
import ctypes

import pytest
import torch

from exact_long_context_tmem_b200 import attn as A
from exact_long_context_tmem_b200 import build as Bld
from tests.parity import device_clean


def test_accept_asks_for_a_path_only_where_there_are_drafts():
    """The check of `path` itself, seen by which error comes first: a call that is refused for its size (more than 65535
    sequences) gets that far without a path if there are no drafts."""
    Bld.build()
    at = [ctypes.c_void_p(0x1000000 * i) for i in range(1, 7)]
    for n_q, status in ((0, A.ATTN_ERR_UNSUPPORTED), (1, A.ATTN_ERR_INVALID_ARG)):
        got = A.lib().attn_tree_accept(at[0], at[1], None, None, 1, 70000, 2, 256, None, 0, 128, 0, at[2], None, n_q,
                                       None, at[3], at[4], None)
        assert got == status


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
def test_accept_of_no_drafts_keeps_the_lengths(cuda_device, paged):
    dev = cuda_device
    k = torch.randn(2, 3, 128, 2, 128, device=dev).to(torch.bfloat16)
    v, kept = k.flip(1).contiguous(), k.clone()
    lens = torch.tensor([128, 0, 77], dtype=torch.int32, device=dev)
    none = torch.zeros(3, dtype=torch.int32, device=dev)
    path = torch.zeros(3, 0, dtype=torch.int32, device=dev)
    table = torch.tensor([[2], [0], [1]], dtype=torch.int32, device=dev) if paged else None
    for q_lens in (None, none):
        out = A.attn_tree_accept(k, v, lens, path, none, q_lens=q_lens, page_table=table)
        assert out.tolist() == [128, 0, 77] and torch.equal(k, kept)
    device_clean()
