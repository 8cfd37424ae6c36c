"""The page oracle on cases worked out by hand, and what the upkeep calls refuse before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

from exact_long_context_tmem_b200 import attn as A
from exact_long_context_tmem_b200 import build as Bld
from oracle import pages as OP
from oracle import tree as OT


def pool(n, page=4):
    return [np.arange(n * page).reshape(1, n, page, 1)]


def test_fork_by_hand():
    # two sequences share page 5; page 2 is cut by children 0 and 1, page 7 goes on in child 2
    c = pool(8)
    t, lens, refs, left = OP.fork(c, [[5, 2], [5, 7]], [7, 6], [0, 0, 1, 0, 0, 2, 0, 1], [0, 0, 1], [6, 7, 6], [9, 7, 6],
                                  4, 4)
    assert t == [[5, 2, 0, -1], [5, 1, -1, -1], [5, 7, -1, -1]]
    assert refs == [1, 1, 1, 0, 0, 3, 0, 1] and left == 3 and lens == [9, 7, 6]
    assert c[0][0, 1, :, 0].tolist() == [8, 9, 10, 7]  # three tokens of page 2


def test_fork_frees_and_refuses():
    c = pool(3)
    t, _, refs, left = OP.fork(c, [[0, 1]], [8], [1, 1, 0], [-1], [0], [4], 4, 2)
    assert t == [[0, -1]] and refs == [1, 0, 0] and left == 2
    assert OP.fork(c, [[0, 1]], [8], [1, 1, 0], [0, -1], [8, 0], [8, 8], 4, 2)[3] == -1


def test_compact_by_hand():
    c = pool(5)
    t, refs, m, n, moved = OP.compact(c, [[4, 1], [1, -1]], [0, 2, 0, 0, 1])
    assert t == [[0, 1], [1, -1]] and refs == [1, 2, 0, 0, 0] and m == [-1, 1, -1, -1, 0] and (n, moved) == (2, 1)
    assert c[0][0, 0, :, 0].tolist() == [16, 17, 18, 19]


def test_accept_reads_before_it_writes():
    c = pool(1, 6)
    OP.accept(c, [1], [[3, 0, 0]], lambda b, s: (b, s))
    assert c[0][0, 0, :, 0].tolist() == [0, 4, 1, 1, 4, 5]


def test_tree_oracle_pins():
    """A full mask row of the drafts' chain is causal attention; a row that sees one slot copies its V."""
    g = np.random.default_rng(1)
    k, v, q = g.normal(size=(1, 9, 1, 4)), g.normal(size=(1, 9, 1, 4)), g.normal(size=(1, 2, 2, 4))
    o, lse = OT.decode_tree(q, k, v, [2], [[1, 2]], scale=0.5)
    np.testing.assert_allclose(o[0, 0], np.stack([v[0, 0, 0]] * 2))
    np.testing.assert_allclose(o[0, 1], np.stack([v[0, 1, 0]] * 2))
    np.testing.assert_allclose(lse[0, 1], 0.5 * q[0, 1] @ k[0, 1, 0])
    from oracle import attention as OA
    want, wl = OA.decode_multi(q, k, v, [9], scale=0.5)
    o, lse = OT.decode_tree(q, k, v, [9], [[1, 3]], scale=0.5)
    np.testing.assert_allclose(o, want)
    np.testing.assert_allclose(lse, wl)
    o, lse = OT.decode_tree(q, k, v, [1], [[0, 3]], scale=0.5, q_lens=[1])
    assert (o == 0).all() and np.isneginf(lse).all()


# ------------------------------------------------------------------------------- refusals

FAKE, MIS = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def L():
    Bld.build()
    return A.lib()


TREE = dict(q=FAKE, k=FAKE, v=FAKE, kv_dtype=0, k_scale=None, v_scale=None, kv_lens=FAKE, q_lens=None, mask=FAKE,
            Tmax=512, n_q=8, dims=A.Dims(2, 8, 2, 128, 0.1), o=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 30)


@pytest.mark.parametrize("case,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(mask=None), 1), (dict(kv_lens=None), 1), (dict(o=None), 1),
    (dict(q=MIS), 1), (dict(v=MIS), 1), (dict(mask=ctypes.c_void_p(0x10004)), 1), (dict(q_lens=ODD), 1),
    (dict(lse=ODD), 1), (dict(Tmax=-1), 1), (dict(n_q=-1), 1), (dict(kv_dtype=2), 1), (dict(kv_dtype=1), 1),
    (dict(k_scale=FAKE, v_scale=FAKE), 1), (dict(ws=None), 1), (dict(ws_bytes=4096), 1), (dict(ws=MIS), 1),
    (dict(dims=A.Dims(2, 7, 2, 128, 0.1)), 1), (dict(dims=A.Dims(2, 8, 2, 128, 0.0)), 1),
    (dict(n_q=65), 2), (dict(dims=A.Dims(2, 8, 2, 96, 0.1)), 2), (dict(dims=A.Dims(2, 258, 2, 128, 0.1)), 2),
    (dict(dims=A.Dims(2, 8, 2, 64, 0.1), kv_dtype=3, k_scale=FAKE, v_scale=FAKE), 2),
    (dict(Tmax=0x7fffffff), 2), (dict(dims=A.Dims(1 << 20, 4096, 4096, 128, 0.1)), 2),
    (dict(dims=A.Dims(0, 8, 2, 128, 0.1), q=None), 0), (dict(n_q=0, q=None), 0),
])
def test_tree_refusals(L, case, status):
    a = dict(TREE, **case)
    got = L.attn_decode_tree(a["q"], a["k"], a["v"], a["kv_dtype"], a["k_scale"], a["v_scale"], a["kv_lens"], a["q_lens"],
                             a["mask"], a["Tmax"], a["n_q"], a["dims"], a["o"], a["lse"], a["ws"], a["ws_bytes"], None)
    assert got == status


@pytest.mark.parametrize("case,status", [(dict(page=100), 1), (dict(page=64), 1), (dict(table=None), 1),
                                         (dict(table=ODD), 1), (dict(max_pages=0), 1), (dict(num_pages=0), 1),
                                         (dict(max_pages=1 << 25), 2)])
def test_tree_paged_refusals(L, case, status):
    a = dict(TREE, table=FAKE, max_pages=4, page=128, num_pages=9)
    a.update(case)
    got = L.attn_decode_tree_paged(a["q"], a["k"], a["v"], 0, None, None, a["table"], a["max_pages"], a["page"],
                                   a["num_pages"], FAKE, None, FAKE, 8, a["dims"], FAKE, None, FAKE, 1 << 30, None)
    assert got == status


def test_tree_workspace_bytes(L):
    assert A.attn_decode_tree_workspace_bytes(2, 8, 2, 128, 0, 8) == 0
    assert A.attn_decode_tree_workspace_bytes(2, 8, 2, 128, 512, 65) == 0
    # two 128-row partials a range, at most one range per (sequence, head, tile)
    assert A.attn_decode_tree_workspace_bytes(1, 8, 2, 128, 256, 8) == 4 * 2 * 128 * 129 * 4


POOL = dict(k=FAKE, v=FAKE, ks=None, vs=None, layers=2, pages=9, page=128, Hkv=2, row=256)


@pytest.mark.parametrize("case,status", [
    (dict(k=None), 1), (dict(v=MIS), 1), (dict(ks=FAKE), 1), (dict(ks=ODD, vs=FAKE), 1), (dict(layers=-1), 1),
    (dict(pages=0), 1), (dict(page=0), 1), (dict(Hkv=0), 1), (dict(row=24), 1), (dict(row=0), 1), (dict(Hkv=1 << 20), 2),
])
def test_pool_refusals(L, case, status):
    a = dict(POOL, **case)
    pool = [a[x] for x in ("k", "v", "ks", "vs", "layers", "pages", "page", "Hkv", "row")]
    assert L.attn_pages_copy(*pool, FAKE, FAKE, 3, None) == status
    assert L.attn_pages_compact(*pool, FAKE, 2, 4, FAKE, ctypes.c_void_p(0x20000), ctypes.c_void_p(0x30000), FAKE, FAKE,
                                None) == status
    out = [ctypes.c_void_p(0x10000 * i) for i in range(2, 6)]
    assert L.attn_pages_fork(*pool, FAKE, FAKE, 2, 4, FAKE, FAKE, FAKE, FAKE, 2, *out, FAKE, 1 << 20, None) == status


def test_upkeep_refusals(L):
    pool = [POOL[x] for x in ("k", "v", "ks", "vs", "layers", "pages", "page", "Hkv", "row")]
    other = ctypes.c_void_p(0x20000)
    assert L.attn_pages_copy(*pool, None, FAKE, 3, None) == 1
    assert L.attn_pages_copy(*pool, FAKE, ODD, 3, None) == 1
    assert L.attn_pages_copy(*pool, FAKE, FAKE, -1, None) == 1
    assert L.attn_pages_copy(*pool, None, None, 0, None) == 0
    big = list(pool)
    big[5] = (1 << 20) + 1
    assert L.attn_pages_copy(*big, FAKE, FAKE, 3, None) == 2
    assert L.attn_pages_compact(*big, FAKE, 2, 4, FAKE, other, other, other, other, None) == 2
    assert L.attn_pages_compact(*pool, FAKE, 2, 4, FAKE, other, FAKE, other, other, None) == 1  # refs in place
    assert L.attn_pages_compact(*pool, FAKE, 2, 4, FAKE, FAKE, other, other, other, None) == 1  # table in place
    f = lambda **k: L.attn_pages_fork(*pool, FAKE, FAKE, 2, k.get("max_pages", 4), FAKE, k.get("parents", FAKE), FAKE,  # noqa: E731
                                      FAKE, k.get("n", 2), k.get("table", other), other, k.get("refs", other), other,
                                      k.get("ws", FAKE), k.get("bytes", 1 << 20), None)
    assert f(parents=None) == 1 and f(table=FAKE) == 1 and f(refs=FAKE) == 1 and f(ws=None) == 1 and f(bytes=64) == 1
    assert f(n=-1) == 1 and f(max_pages=0) == 1 and f(n=1 << 20, max_pages=1 << 11, bytes=1 << 40) == 2
    assert A.attn_pages_fork_workspace_bytes(3, 100) == (12 + 100 + 4) * 4
    acc = lambda **k: L.attn_tree_accept(FAKE, FAKE, None, None, k.get("layers", 1), k.get("B", 2), 2, 256,  # noqa: E731
                                         k.get("table"), 4, k.get("page", 128), 9, FAKE, None, k.get("n_q", 8),
                                         k.get("path", FAKE), FAKE, k.get("out", other), None)
    assert acc(path=None) == 1 and acc(out=FAKE) == 1 and acc(out=None) == 1 and acc(layers=0) == 1
    assert acc(table=FAKE, page=100) == 1 and acc(n_q=65) == 2 and acc(B=70000) == 2 and acc(B=0) == 0


def test_binding_refuses_host_tensors():
    k = torch.zeros(1, 2, 128, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: A.attn_pages_copy(k, k, i, i), lambda: A.attn_tree_accept(k, k, i, i[:, None], i),
                 lambda: A.attn_pages_compact(k, k, i[:, None], i),
                 lambda: A.attn_decode_tree(k[0, :, :4], k[0], k[0], i, i[:, None].long())):
        with pytest.raises(ValueError, match="device tensors"):
            call()


def test_cache_shapes_are_checked():
    k = torch.zeros(1, 2, 128, 2, 128, dtype=torch.bfloat16)
    assert A._cache(k, k, None, None) == (1, 2, 128, 2, 256)
    assert A._cache(k[0], k[0], None, None) == (1, 2, 128, 2, 256)
    c, s = k.to(torch.int8), torch.zeros(1, 2, 128, 2)
    assert A._cache(c, c, s, s) == (1, 2, 128, 2, 128)
    for bad in ((k, k[:, :1], None, None), (c, c, None, None), (k, k, s, s), (k.float(), k.float(), None, None),
                (c, c, s, s[..., :1]), (k.transpose(1, 2), k.transpose(1, 2), None, None), (k[0, 0], k[0, 0], None, None),
                (k[:, :0], k[:, :0], None, None)):
        with pytest.raises(ValueError):
            A._cache(*bad)
