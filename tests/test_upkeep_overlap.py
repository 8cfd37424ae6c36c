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


PAGES, CHILDREN = 12, 3
ROOM = {name: (0x100000 * (i + 1), n) for i, (name, n) in enumerate([
    ("table", B * MAX_PAGES), ("kv_lens", B), ("refs", PAGES), ("parents", CHILDREN), ("keep", CHILDREN),
    ("new", CHILDREN), ("table_out", CHILDREN * MAX_PAGES), ("lens_out", CHILDREN), ("refs_out", PAGES), ("info", 2),
    ("ws", CHILDREN * 4 + PAGES + 4), ("map", PAGES), ("big_out", B * MAX_PAGES)])}


def pool_call(L, call, at):
    p = {x: ctypes.c_void_p(at.get(x, a)) for x, (a, _) in ROOM.items()}
    pool = [ctypes.c_void_p(0x10000000), ctypes.c_void_p(0x20000000), None, None, 1, PAGES, 128, 2, 256]
    if call == "fork":
        return L.attn_pages_fork(*pool, p["table"], p["kv_lens"], B, MAX_PAGES, p["refs"], p["parents"], p["keep"],
                                 p["new"], CHILDREN, p["table_out"], p["lens_out"], p["refs_out"], p["info"], p["ws"],
                                 1 << 20, None)
    return L.attn_pages_compact(*pool, p["table"], B, MAX_PAGES, p["refs"], p["big_out"], p["refs_out"], p["map"],
                                p["info"], None)


@pytest.mark.parametrize("call,out", [("fork", x) for x in ("table_out", "lens_out", "refs_out", "info", "ws")] +
                         [("compact", x) for x in ("big_out", "refs_out", "map", "info")])
def test_pool_calls_refuse_outputs_over_other_arrays(L, call, out):
    assert A.attn_pages_fork_workspace_bytes(CHILDREN, PAGES) == 4 * ROOM["ws"][1]
    fork = ("table", "kv_lens", "refs", "parents", "keep", "new", "table_out", "lens_out", "refs_out", "info", "ws")
    for other in fork if call == "fork" else ("table", "refs", "big_out", "refs_out", "map", "info"):
        if other == out:
            continue
        at, n = ROOM[other]
        for shift in (0, n - 1, 1 - ROOM[out][1]):
            assert pool_call(L, call, {out: at + 4 * shift}) == A.ATTN_ERR_INVALID_ARG, (other, shift)


def test_overlap_of_tensors():
    x = torch.zeros(32, dtype=torch.int32)
    assert A._overlap(x, x) and A._overlap(x[3:9], x[8:20]) and A._overlap(x[8:20], x[3:9])
    assert not A._overlap(x[:8], x[8:]) and not A._overlap(x[8:], x[:8])
    assert not A._overlap(x, None) and not A._overlap(x[:0], x)
