"""Compaction of a pool whose counts are corrupt: nothing may move over a page that somebody's table still names."""
import random

import pytest
import torch

from exact_long_context_tmem_b200 import attn as A
from oracle import pages as OP
from tests.parity import device_clean
from tests.test_gpu_pages import as_bytes, ints, make_cache, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("N,at", [(5, 0), (131, 130), (4096, 77), (4096, 4095)])
def test_a_negative_count_moves_nothing(cuda_device, kind, N, at):
    dev, r = cuda_device, random.Random(N)
    refs = [r.choice([0, 0, 1, 2]) for _ in range(N)]
    refs[-1], refs[at] = 1, -1
    live = [p for p in range(N) if refs[p] > 0]
    table = [[p for p in r.sample(live, min(len(live), 20))] + [at, -1] for _ in range(7)]
    width = max(map(len, table))
    table = [x + [-1] * (width - len(x)) for x in table]
    caches = make_cache(kind, (2, N, 128), 1, 3, dev)
    k, v, ks, vs = caches
    want = as_bytes(caches)
    args = ints(table, dev), ints(refs, dev)
    t, f, m, info = A.attn_pages_compact(k, v, *args, k_scale=ks, v_scale=vs)
    assert same(caches, want)
    assert t.tolist() == table and f.tolist() == refs and m.tolist() == list(range(N)) and info.tolist() == [-1, 0]
    assert A.attn_device_status(reset=True) == (A.ATTN_ERR_INVALID_ARG, 72)
    refs[at] = 0  # and with the count put right the call compacts
    t, f, m, info = A.attn_pages_compact(k, v, args[0], ints(refs, dev), k_scale=ks, v_scale=vs)
    wt, wf, wm, n_live, moved = OP.compact(want, table, refs)
    assert t.tolist() == wt and f.tolist() == wf and m.tolist() == wm and info.tolist() == [n_live, moved]
    assert all((a[:, :n_live] == b[:, :n_live]).all() for a, b in zip(as_bytes(caches), want, strict=True))
    device_clean()
