"""Calls of the tree decode and the upkeep that are allowed and rarely made: nobody there, more sequences than processors
by far, lengths past either end, the widest groups over coded caches."""
import numpy as np
import pytest
import torch

from exact_long_context_tmem_b200 import attn as A
from tests.parity import device_clean
from tests.test_gpu_pages import as_bytes, ints, make_cache, same
from tests.test_gpu_tree import KINDS, check, make, tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("n_q,Hq,Hkv", [(5, 128, 1), (64, 128, 1), (3, 200, 2), (1, 128, 1)])
def test_widest_groups(cuda_device, kind, n_q, Hq, Hkv):
    d = make(kind, 2, n_q, Hq, Hkv, [max(n_q, 300), n_q], 320, seed=n_q)
    check(*tree(d, kind, cuda_device), d, kind)
    device_clean()


@pytest.mark.parametrize("kind", list(KINDS))
def test_thousands_of_short_sequences(cuda_device, kind):
    g = np.random.default_rng(8)
    B, n_q = 3000, 6
    q_lens = g.integers(0, n_q + 1, size=B).tolist()
    lens = [max(q, int(x)) for q, x in zip(q_lens, g.integers(0, 200, size=B))]
    d = make(kind, B, n_q, 4, 1, lens, 200, seed=1)
    o, lse = tree(d, kind, cuda_device, q_lens=q_lens)
    again = tree(d, kind, cuda_device, q_lens=q_lens)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    pick = [0, 1, 2, 1499, 1500, 2998, 2999] + g.integers(0, B, size=40).tolist()
    sub = {x: (y[pick] if isinstance(y, torch.Tensor) else y) for x, y in d.items()}
    check(o[pick], lse[pick], sub, kind, q_lens=[q_lens[b] for b in pick])
    device_clean()


@pytest.mark.parametrize("kind", list(KINDS))
def test_lengths_past_either_end_are_clamped(cuda_device, kind):
    d = make(kind, 5, 7, 8, 2, [300, 300, 300, 300, 300], 300, seed=2)
    given = [300, 1 << 30, -4, 300, -(1 << 31)]
    q_given = [7, 99, 7, -3, 7]
    want = tree(dict(d, kv_lens=torch.tensor([300, 300, 0, 300, 0], dtype=torch.int32)), kind, cuda_device,
                q_lens=[7, 7, 7, 0, 7])
    got = tree(dict(d, kv_lens=torch.tensor(given, dtype=torch.int32)), kind, cuda_device, q_lens=q_given)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert torch.isneginf(got[1][2:]).all() and (got[0][2:] == 0).all()
    device_clean()


def test_nobody(cuda_device):
    """No sequences before or after, no pages to copy, no table to rewrite."""
    dev = cuda_device
    caches = make_cache("fp8", (2, 9, 128), 2, 1, dev)
    k, v, ks, vs = caches
    want, sc = as_bytes(caches), dict(k_scale=ks, v_scale=vs)
    none = ints([], dev)
    empty = torch.empty(0, 3, dtype=torch.int32, device=dev)
    refs = ints([0, 2, 0, 0, 1, 0, 0, 0, 0], dev)  # pinned pages
    # admission into an empty pool
    t, l, f, info = A.attn_pages_fork(k, v, empty, none, refs, ints([-1, -1], dev), keep_lens=ints([5, 0], dev),
                                      new_lens=ints([130, 0], dev), **sc)
    assert t.tolist() == [[0, 2, -1], [-1, -1, -1]] and l.tolist() == [130, 0] and info.tolist() == [5, 0]
    assert f.tolist() == [1, 2, 1, 0, 1, 0, 0, 0, 0]
    # everybody ends
    t2, l2, f2, info = A.attn_pages_fork(k, v, t, l, f, none, keep_lens=none, new_lens=none, **sc)
    assert t2.shape == (0, 3) and l2.numel() == 0 and f2.tolist() == refs.tolist() and info.tolist() == [7, 0]
    A.attn_pages_copy(k, v, none, none, **sc)
    assert same(caches, want)
    t, f, m, info = A.attn_pages_compact(k, v, empty, refs, **sc)
    assert t.shape == (0, 3) and f.tolist() == [1, 2] + [0] * 7 and info.tolist() == [2, 1]
    assert m.tolist() == [-1, 1, -1, -1, 0, -1, -1, -1, -1]
    o, lse = A.attn_decode_tree(torch.empty(0, 4, 8, 128, dtype=torch.bfloat16, device=dev), k[0, :0], v[0, :0], none,
                                torch.empty(0, 4, dtype=torch.int64, device=dev), k_scale=ks[0, :0], v_scale=vs[0, :0])
    assert o.shape == (0, 4, 8, 128) and lse.shape == (0, 4, 8)
    device_clean()


def test_queries_and_outputs_in_one_place(cuda_device):
    """o may be q: a row block's queries are read by the CTA that writes it, or before the join does."""
    for n_q, G, lens in ((6, 4, [700, 90, 2000]), (40, 4, [1500] * 5), (64, 16, [900, 64])):
        d = make("bf16", len(lens), n_q, 2 * G, 2, lens, 2048, seed=G)
        want, _ = tree(d, "bf16", cuda_device)
        dev = cuda_device
        q = d["q"].to(dev)
        A.attn_decode_tree(q, d["k"].to(dev), d["v"].to(dev), d["kv_lens"].to(dev), d["mask"].to(dev), o=q)
        assert torch.equal(q, want)
    device_clean()
