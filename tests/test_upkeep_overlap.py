"""Outputs of the upkeep calls that overlap what the same call reads are refused before any CUDA call.

The addresses below are never read: every call of this file is refused, or has nothing to do.
"""
import ctypes

import pytest
import torch

from exact_long_context_tmem_b200 import attn as A
from exact_long_context_tmem_b200 import build as Bld

B, N_Q, MAX_PAGES = 6, 8, 4
AT = {name: 0x100000 * (i + 1) for i, name in enumerate(
    ("k", "v", "kv_lens", "q_lens", "path", "n_accepted", "table", "out"))}


@pytest.fixture(scope="module")
def L():
    Bld.build()
    return A.lib()


def accept(L, at):
    p = {x: ctypes.c_void_p(y) for x, y in {**AT, **at}.items()}
    return L.attn_tree_accept(p["k"], p["v"], None, None, 1, B, 2, 256, p["table"], MAX_PAGES, 128, 9, p["kv_lens"],
                              p["q_lens"], N_Q, p["path"], p["n_accepted"], p["out"], None)


@pytest.mark.parametrize("name,length", [("kv_lens", B), ("q_lens", B), ("n_accepted", B), ("path", B * N_Q),
                                         ("table", B * MAX_PAGES)])
def test_accept_refuses_lengths_over_its_inputs(L, name, length):
    for shift in (0, 1, -1, length - 1, 1 - B):  # in elements: the same place, and overlaps at either end
        assert accept(L, {"out": AT[name] + 4 * shift}) == A.ATTN_ERR_INVALID_ARG, shift


def test_overlap_of_tensors():
    x = torch.zeros(32, dtype=torch.int32)
    assert A._overlap(x, x) and A._overlap(x[3:9], x[8:20]) and A._overlap(x[8:20], x[3:9])
    assert not A._overlap(x[:8], x[8:]) and not A._overlap(x[8:], x[:8])
    assert not A._overlap(x, None) and not A._overlap(x[:0], x)
