"""Many speculation steps over one pool: drafts cross page borders and are rejected, and no page is lost.

The lengths that a generation's pages are held for are those attn_pages_fork gave out; attn_tree_accept shortens
the sequences, not what they hold.  So the next fork takes the former as kv_lens and the latter as keep_lens."""
import random

import pytest
import torch

from exact_long_context_tmem_b200 import attn as A
from tests.parity import device_clean
from tests.test_gpu_pages import ints

pytestmark = pytest.mark.gpu


def counts(table, N):
    out = [0] * N
    for row in table.tolist():
        for p in row:
            if p >= 0:
                out[p] += 1
    return out


@pytest.mark.parametrize("n_q", [5, 64])
@pytest.mark.parametrize("compact", [False, True])
def test_a_pool_survives_many_steps(cuda_device, n_q, compact):
    dev, page, B, N, width, steps = cuda_device, 128, 6, 64, 10, 30
    r = random.Random(n_q)
    k = torch.zeros(1, N, page, 1, 64, dtype=torch.bfloat16, device=dev)
    v = torch.zeros_like(k)
    start = [r.randint(1, 200) for _ in range(B)]
    none = ints([], dev)
    table, held, refs, info = A.attn_pages_fork(
        k, v, torch.empty(0, width, dtype=torch.int32, device=dev), none, torch.zeros(N, dtype=torch.int32, device=dev),
        ints([-1] * B, dev), keep_lens=ints([0] * B, dev), new_lens=ints(start, dev))
    lens, want = held, list(start)  # what the sequences are, against what they hold pages for
    mark = torch.zeros(B, width * page, device=dev)  # what their tokens are, by hand
    slots = torch.arange(width * page, device=dev)

    def at(b, lo, hi):
        s = slots[lo:hi]
        return table[b].long()[s // page], s % page
    for b, n in enumerate(start):
        mark[b, :n] = torch.arange(n, device=dev) % 199 + 256 * (b == 0)
        k[0, at(b, 0, n)[0], at(b, 0, n)[1]] = mark[b, :n, None, None].to(torch.bfloat16)
    for step in range(steps):
        table, held, refs, info = A.attn_pages_fork(k, v, table, held, refs, ints(list(range(B)), dev), keep_lens=lens,
                                                    new_lens=lens + n_q)
        assert info[1] == 0 and refs.tolist() == counts(table, N)
        assert int(info[0]) == sum(x == 0 for x in refs.tolist())
        assert int((table >= 0).sum()) == sum(-(-(n + n_q) // page) for n in want)
        path, acc = [], []
        for b, n in enumerate(want):
            draft = torch.arange(n_q, device=dev) + 1.0 + step
            k[0, at(b, n, n + n_q)[0], at(b, n, n + n_q)[1]] = draft[:, None, None].to(torch.bfloat16)
            a = r.choice([0, 1, r.randint(0, min(n_q, 30))])
            path.append(sorted(r.sample(range(n_q), a)))
            acc.append(a)
            mark[b, n:n + a] = draft[path[b]]
        lens = A.attn_tree_accept(k, v, held, ints([p + [0] * (n_q - len(p)) for p in path], dev), ints(acc, dev),
                                  page_table=table)
        want = [n + a for n, a in zip(want, acc)]
        assert lens.tolist() == want
        if compact:
            table, refs, _, _ = A.attn_pages_compact(k, v, table, refs)
        for b, n in enumerate(want):
            pg, off = at(b, 0, n)
            assert torch.equal(k[0, pg, off, 0, 0], mark[b, :n].to(torch.bfloat16))
        over = [b for b, n in enumerate(want) if n + 2 * n_q > (width - 1) * page]
        if over:  # a sequence ends and another begins in its place
            new = [min(n, 100) if b in over else n for b, n in enumerate(want)]
            table, held, refs, info = A.attn_pages_fork(k, v, table, held, refs, ints(list(range(B)), dev),
                                                        keep_lens=ints(new, dev), new_lens=ints(new, dev))
            lens, want = held, new
            assert info[1] == 0 and refs.tolist() == counts(table, N)
    _, _, refs, info = A.attn_pages_fork(k, v, table, held, refs, none, keep_lens=none, new_lens=none)
    assert refs.tolist() == [0] * N and info.tolist() == [N, 0]
    device_clean()
