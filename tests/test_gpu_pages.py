"""The upkeep of a cache on the GPU, compared byte by byte with oracle/pages.py."""
import random

import numpy as np
import pytest
import torch

from exact_long_context_tmem_b200 import attn as A
from oracle import pages as OP
from tests.parity import device_clean

pytestmark = pytest.mark.gpu

# element type, bytes of a row with D = 128, scales
KINDS = {"bf16": (torch.bfloat16, 128, False), "fp8": (torch.uint8, 128, True), "int8": (torch.int8, 128, True),
         "int4": (torch.uint8, 64, True)}


def make_cache(kind, lead, Hkv, seed, dev):
    """Random bytes: K, V (and scales) of shape [*lead, Hkv, row]."""
    dtype, row, coded = KINDS[kind]
    g = torch.Generator().manual_seed(seed)
    def ints(last, dt):
        size = torch.empty(0, dtype=dt).element_size()
        x = torch.randint(0, 256, (*lead, Hkv, last * size), generator=g, dtype=torch.uint8)
        return x.view(dt).to(dev)
    k, v = ints(row, dtype), ints(row, dtype)
    if not coded:
        return k, v, None, None
    return k, v, ints(1, torch.float32)[..., 0].contiguous(), ints(1, torch.float32)[..., 0].contiguous()


def as_bytes(caches):
    """Host copies as bytes, [layers, pages, tokens, bytes]."""
    out = []
    for x in caches:
        if x is not None:
            y = x.cpu()
            if y.dtype == torch.bfloat16:
                y = y.view(torch.int16)
            y = np.ascontiguousarray(y.numpy())
            out.append(y.view(np.uint8).reshape(*y.shape[:3], -1))
    return out


def same(caches, want):
    return all(np.array_equal(a, b) for a, b in zip(as_bytes(caches), want, strict=True))


def ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


# ------------------------------------------------------------------------------- accepted path

@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("Hkv,layers", [(8, 1), (5, 3), (1, 2)])
def test_accept(cuda_device, kind, paged, Hkv, layers):
    dev, r = cuda_device, random.Random(Hkv + layers)
    B, n_q, T, page = 6, 40, 300, 128
    q_lens = [40, 40, 7, 0, 1, 40]
    lens = [300, 40, 300, 12, 1, 129 + 20]  # the last one's drafts lie on both sides of a page's end
    path = [sorted(r.sample(range(40), 17)), list(range(40)), [], [], [0],
            [39, 3, 3, 0, 17]]  # falling, with a repeat
    per = -(-T // page)
    order = r.sample(range(B * per + 2), B * per)
    table = [order[b * per:(b + 1) * per] for b in range(B)]
    lead = (layers, B * per + 2, page) if paged else (layers, B, T)
    caches = make_cache(kind, lead, Hkv, 3, dev)
    want = as_bytes(caches)
    base = [n - q for n, q in zip(lens, q_lens)]
    rows = (lambda b, s: (table[b][s // page], s % page)) if paged else (lambda b, s: (b, s))
    OP.accept(want, base, path, rows)
    k, v, ks, vs = caches
    out = A.attn_tree_accept(k, v, ints(lens, dev), ints([x + [-5] * (n_q - len(x)) for x in path], dev),
                             ints([len(x) for x in path], dev), q_lens=ints(q_lens, dev), k_scale=ks, v_scale=vs,
                             page_table=ints(table, dev) if paged else None)
    assert same(caches, want)
    assert out.tolist() == [b + len(x) for b, x in zip(base, path)]
    device_clean()


def test_accept_one_layer_without_its_dimension(cuda_device):
    dev = cuda_device
    k, v, _, _ = make_cache("bf16", (1, 2, 64), 2, 1, dev)
    want = as_bytes((k, v))
    OP.accept(want, [60, 10], [[1, 3], [2]], lambda b, s: (b, s))
    out = A.attn_tree_accept(k[0], v[0], ints([64, 14], dev), ints([[1, 3, 0, 0], [2, 0, 0, 0]], dev), ints([2, 1], dev))
    assert same((k, v), want) and out.tolist() == [62, 11]
    device_clean()


def test_accept_writes_the_lengths_where_it_is_told(cuda_device):
    dev = cuda_device
    k, v, _, _ = make_cache("bf16", (1, 2, 64), 2, 1, dev)
    lens, path, n = ints([64, 14], dev), ints([[1, 3, 0, 0], [2, 0, 0, 0]], dev), ints([2, 1], dev)
    with pytest.raises(ValueError, match="kv_lens_out"):
        A.attn_tree_accept(k[0], v[0], lens, path, n, kv_lens_out=lens)
    with pytest.raises(ValueError, match="kv_lens"):
        A.attn_tree_accept(k[0], v[0], lens[0], path[:1], n[:1])
    room = ints([-7, -7, -7], dev)
    out = A.attn_tree_accept(k[0], v[0], lens, path, n, kv_lens_out=room[:2])
    assert out.data_ptr() == room.data_ptr() and room.tolist() == [62, 11, -7] and lens.tolist() == [64, 14]
    device_clean()


@pytest.mark.parametrize("bad", ["draft", "count", "length", "page", "negative"])
def test_accept_leaves_a_bad_sequence_alone(cuda_device, bad):
    dev = cuda_device
    k, v, ks, vs = caches = make_cache("int8", (2, 6, 128), 4, 1, dev)
    lens, n_acc, path, table = [200, 100, 256], [3, 2, 4], [[1, 2, 5, 0], [0, 3, 0, 0], [2, 3, 4, 7]], [[0, 1], [2, 3], [4, 5]]
    n_q = 8
    path = [x + [0] * 4 for x in path]
    if bad == "draft":
        path[0][1] = 8
    elif bad == "negative":
        path[0][1] = -1
    elif bad == "count":
        n_acc[0] = 9
    elif bad == "length":
        lens[0] = 7
    else:
        table[0][1] = 6
    want = as_bytes(caches)
    OP.accept(want, [0, 92, 248], [[], path[1][:2], path[2][:4]], lambda b, s: (table[b][s // 128], s % 128))
    out = A.attn_tree_accept(k, v, ints(lens, dev), ints(path, dev), ints(n_acc, dev), n_q=n_q, k_scale=ks, v_scale=vs,
                             page_table=ints(table, dev))
    assert same(caches, want) and out.tolist() == [lens[0], 94, 252]
    assert A.attn_device_status(reset=True) == (A.ATTN_ERR_INVALID_ARG, 70)


# ------------------------------------------------------------------------------- copies

@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("Hkv,layers,pages,n", [(1, 1, 2, 1), (5, 3, 70, 33), (8, 2, 40, 20)])
def test_copy(cuda_device, kind, Hkv, layers, pages, n):
    dev, r = cuda_device, random.Random(n)
    caches = make_cache(kind, (layers, pages, 128), Hkv, 2, dev)
    order = r.sample(range(pages), 2 * n)
    src, dst = order[:n], order[n:]
    src[n // 2] = src[0]  # one page to several places
    want = as_bytes(caches)
    OP.copy_pages(want, src, dst)
    k, v, ks, vs = caches
    A.attn_pages_copy(k, v, ints(src, dev), ints(dst, dev), k_scale=ks, v_scale=vs)
    assert same(caches, want)
    device_clean()


@pytest.mark.parametrize("src,dst", [([0, 1], [2, 2]), ([0, 2], [2, 3]), ([0, 1], [1, 0]), ([9, 1], [2, 3]),
                                     ([0, 1], [2, 8]), ([-1, 1], [2, 3])])
def test_copy_refuses_lists_without_one_answer(cuda_device, src, dst):
    dev = cuda_device
    caches = make_cache("fp8", (2, 8, 128), 2, 2, dev)
    want = as_bytes(caches)
    k, v, ks, vs = caches
    A.attn_pages_copy(k, v, ints(src, dev), ints(dst, dev), k_scale=ks, v_scale=vs)
    assert same(caches, want)
    assert A.attn_device_status(reset=True) == (A.ATTN_ERR_INVALID_ARG, 71)
    A.attn_pages_copy(k, v, ints([3, 4], dev), ints([3, 5], dev), k_scale=ks, v_scale=vs)  # 3 -> 3 does nothing
    OP.copy_pages(want, [4], [5])
    assert same(caches, want)
    device_clean()


# ------------------------------------------------------------------------------- fork and compact

def random_pool(r, B, page, T, spare, pins=0):
    """Sequences over a pool in random order with shared prefixes, and their reference counts."""
    width = T // page + 3
    N = B * (T // page + 2) + spare
    order = r.sample(range(N), N)
    lens, table, refs = [], [], [0] * N
    for b in range(B):
        n = r.choice([0, 1, page, r.randint(1, T), r.randint(1, T), T])
        held = -(-n // page)
        row = []
        if b and r.random() < 0.6:
            o = r.randrange(b)
            row = table[o][:r.randint(0, min(lens[o], n) // page)]
        row = row + [order.pop() for _ in range(held - len(row))]
        for p in row:
            refs[p] += 1
        lens.append(n)
        table.append(row)
    for _ in range(pins):
        refs[r.randrange(N)] += 1
    return lens, table, refs, width, N


def random_children(r, lens, n, page, width):
    parents, keep, new = [], [], []
    for c in range(n):
        a = r.choice([-1, r.randrange(len(lens)), r.randrange(len(lens)), c % len(lens)])
        k = r.choice([0, -3, page, r.randint(0, width * page), (lens[a] if a >= 0 else 0), 10**9])
        parents.append(a)
        keep.append(k)
        new.append(r.choice([0, r.randint(0, (width - 1) * page), max(0, min(k, lens[a] if a >= 0 else 0)) + r.choice([0, 1, 40])]))
    return parents, keep, new


def pad(rows, width, dev):
    return ints([x + [-1] * (width - len(x)) for x in rows], dev).reshape(len(rows), width)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("seed", range(6))
def test_fork(cuda_device, kind, seed):
    dev, r = cuda_device, random.Random(seed)
    page, B = r.choice([128, 256]), r.choice([1, 5, 40])
    lens, table, refs, width, N = random_pool(r, B, page, 900, r.choice([40, 300]), pins=r.choice([0, 3]))
    caches = make_cache(kind, (r.choice([1, 3]), N, page), r.choice([1, 3, 4]), seed, dev)
    k, v, ks, vs = caches
    want = as_bytes(caches)
    args = pad(table, width, dev), ints(lens, dev), ints(refs, dev)
    kept = [x.clone() for x in args]
    for _ in range(3):  # a few generations in a row
        n = r.choice([1, B, B + 3])
        parents, keep, new = random_children(r, lens, n, page, width)
        got = A.attn_pages_fork(k, v, *args, ints(parents, dev), keep_lens=ints(keep, dev), new_lens=ints(new, dev),
                                k_scale=ks, v_scale=vs)
        t, l, f, left = OP.fork(want, table, lens, refs, parents, keep, new, page, width)
        assert all(torch.equal(a, b) for a, b in zip(args, kept))  # the old generation is not written
        assert same(caches, want)
        if t is None:
            assert got[3].tolist() == [left, A.ATTN_ERR_BUDGET]
            assert (got[0] == -1).all() and (got[1] == 0).all() and got[2].tolist() == refs
            continue
        assert got[0].tolist() == t and got[1].tolist() == l and got[2].tolist() == f
        assert got[3].tolist() == [left, 0]
        args, kept = got[:3], [x.clone() for x in got[:3]]
        table, lens, refs = [[p for p in row if p >= 0] for row in t], l, f
    device_clean()


def test_fork_of_a_large_pool(cuda_device):
    """More pages than shared memory counts: the tables are kept in the workspace."""
    dev, r = cuda_device, random.Random(5)
    page, N, B, width = 128, 26000, 300, 60
    order = r.sample(range(N), N)
    lens = [r.randint(0, 58 * page) for _ in range(B)]
    table = [[order.pop() for _ in range(-(-n // page))] for n in lens]
    refs = [0] * N
    for row in table:
        for p in row:
            refs[p] += 1
    caches = make_cache("int4", (1, N, page), 1, 1, dev)
    k, v, ks, vs = caches
    want = as_bytes(caches)
    parents, keep, new = random_children(r, lens, B, page, width)
    got = A.attn_pages_fork(k, v, pad(table, width, dev), ints(lens, dev), ints(refs, dev), ints(parents, dev),
                            keep_lens=ints(keep, dev), new_lens=ints(new, dev), k_scale=ks, v_scale=vs)
    t, l, f, left = OP.fork(want, table, lens, refs, parents, keep, new, page, width)
    assert t is not None
    assert got[0].tolist() == t and got[1].tolist() == l and got[2].tolist() == f and got[3].tolist() == [left, 0]
    assert same(caches, want)
    device_clean()


@pytest.mark.parametrize("bad", ["parent", "new_len", "len", "entry", "count"])
def test_fork_refuses_bad_tables(cuda_device, bad):
    dev = cuda_device
    caches = make_cache("bf16", (1, 9, 128), 2, 1, dev)
    k, v, _, _ = caches
    want = as_bytes(caches)
    table, lens, refs, parents, keep, new = [[0, 1], [0, 2]], [130, 250], [2, 1, 1] + [0] * 6, [0, 1], [130, 5], [140, 9]
    if bad == "parent":
        parents[1] = 2
    elif bad == "new_len":
        new[0] = 3 * 128 + 1
    elif bad == "len":
        lens[1] = -1
    elif bad == "entry":
        table[1][0] = 9
    else:
        refs[0] = 1
    got = A.attn_pages_fork(k, v, pad(table, 3, dev), ints(lens, dev), ints(refs, dev), ints(parents, dev),
                            keep_lens=ints(keep, dev), new_lens=ints(new, dev))
    assert got[3].tolist()[1] == A.ATTN_ERR_INVALID_ARG and (got[0] == -1).all() and got[2].tolist() == refs
    assert same(caches, want)
    assert A.attn_device_status(reset=True) == (A.ATTN_ERR_INVALID_ARG, 73)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("seed", range(5))
def test_compact(cuda_device, kind, seed):
    dev, r = cuda_device, random.Random(seed)
    page = 128
    lens, table, refs, width, N = random_pool(r, r.choice([1, 9, 40]), page, 900, r.choice([0, 1, 77, 400]),
                                              pins=r.choice([0, 2]))
    if seed == 3:
        refs = [0] * N  # nobody left
    if seed == 4:
        refs = [1 + x for x in refs]  # nothing free
    caches = make_cache(kind, (r.choice([1, 3]), N, page), r.choice([1, 3]), seed, dev)
    k, v, ks, vs = caches
    want = as_bytes(caches)
    got = A.attn_pages_compact(k, v, pad(table, width, dev), ints(refs, dev), k_scale=ks, v_scale=vs)
    t, f, m, n_live, moved = OP.compact(want, table, refs)
    assert got[0].tolist() == [x + [-1] * (width - len(x)) for x in t]
    assert got[1].tolist() == f and got[2].tolist() == m and got[3].tolist() == [n_live, moved]
    for a, b in zip(as_bytes(caches), want, strict=True):  # free pages may hold anything, and are left as they were
        assert np.array_equal(a[:, :n_live], b[:, :n_live])
    device_clean()


def test_compact_reports_a_bad_entry(cuda_device):
    dev = cuda_device
    k, v, _, _ = make_cache("bf16", (1, 5, 128), 1, 1, dev)
    t, f, m, info = A.attn_pages_compact(k, v, ints([[4, 7, -1, 2]], dev), ints([0, 0, 1, 0, 1], dev))
    assert t.tolist() == [[1, -1, -1, 0]] and m.tolist() == [-1, -1, 0, -1, 1] and f.tolist() == [1, 1, 0, 0, 0]
    assert info.tolist() == [2, 2]
    assert A.attn_device_status(reset=True) == (A.ATTN_ERR_INVALID_ARG, 72)


# ------------------------------------------------------------------------------- together

@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_speculation_over_a_pool(cuda_device, kind):
    """Prompts shared by two beams each; every step forks them with room for drafts, verifies a tree, keeps a
    path; then the pool is compacted.  After it all, a decode over the pool equals one over a contiguous
    cache built by hand, and the whole run, captured in a graph and replayed, repeats it."""
    dev, page, n_q, Hq, Hkv, N, width = cuda_device, 128, 6, 8, 2, 48, 6
    g = torch.Generator().manual_seed(1)
    r = random.Random(2)
    coded = kind == "fp8"

    def rows(*lead):
        if not coded:
            return [torch.randn(*lead, Hkv, 128, generator=g).to(torch.bfloat16).to(dev) for _ in range(2)] + [None] * 2
        codes = [torch.randint(0, 120, (*lead, Hkv, 128), generator=g, dtype=torch.uint8).to(dev) for _ in range(2)]
        return codes + [(0.005 * (1 + torch.rand(*lead, Hkv, generator=g))).to(dev) for _ in range(2)]

    pool = rows(1, N, page)
    lens, table, refs = [300, 250], [[11, 4, 40], [7, 30]], [0] * N
    for row in table:
        for p in row:
            refs[p] += 1
    start = pad(table, width, dev), ints(lens, dev), ints(refs, dev)
    contig = [None if x is None else torch.stack([x[0, t].flatten(0, 1)[:256] for t in
              (torch.tensor([11, 4], device=dev), torch.tensor([7, 30], device=dev))]) for x in pool]
    steps = []
    for i in range(3):
        path = [sorted(r.sample(range(n_q), 3)) for _ in range(4)]
        draft = rows(4, n_q)
        mask = torch.tensor([[(1 << (j + 1)) - 1 for j in range(n_q)]] * 4, dtype=torch.int64, device=dev)
        q = torch.randn(4, n_q, Hq, 128, generator=g).to(torch.bfloat16).to(dev)
        acc = ints([3, 1, 2, 0], dev)
        steps.append((ints([x + [0] * 3 for x in path], dev), draft, mask, q, acc, path))
    q1 = torch.randn(4, Hq, 128, generator=g).to(torch.bfloat16).to(dev)
    par = [ints([0, 0, 1, 1], dev)] + [ints([0, 1, 2, 3], dev)] * 2
    slot = torch.arange(n_q, device=dev)
    kept = [None if x is None else x.clone() for x in pool]

    def run():
        sc = dict(k_scale=pool[2], v_scale=pool[3])
        t, l, f = start
        outs = []
        for i, (path, draft, mask, q, acc, _) in enumerate(steps):
            old = l[par[i].long()]
            t, l, f, info = A.attn_pages_fork(pool[0], pool[1], t, l, f, par[i], keep_lens=old, new_lens=old + n_q, **sc)
            at = (l[:, None] - n_q + slot).long()
            pg = t.gather(1, at // page).long()
            for x, y in zip(pool, draft):
                if x is not None:
                    x[0, pg, at % page] = y
            one = dict(k_scale=pool[2][0], v_scale=pool[3][0]) if coded else {}
            o, lse = A.attn_decode_tree_paged(q, pool[0][0], pool[1][0], t, l, mask, **one)
            l = A.attn_tree_accept(pool[0], pool[1], l, path, acc, page_table=t, **sc)
            outs += [o, lse, info]
        t, f, m, info = A.attn_pages_compact(pool[0], pool[1], t, f, **sc)
        one = dict(k_scale=pool[2][0], v_scale=pool[3][0]) if coded else {}
        o, lse = A.attn_decode_paged(q1, pool[0][0], pool[1][0], t, l, **one)
        return outs + [o, lse, t, l, f, info]

    got = [x.clone() for x in run()]
    after = [None if x is None else x.clone() for x in pool]
    assert got[-3].tolist() == [300 + 9, 300 + 3, 250 + 6, 250]
    # the same history by hand, contiguous
    prompt = [torch.tensor(p, device=dev) for p in ([11, 4, 40], [11, 4, 40], [7, 30], [7, 30])]
    T = 400
    hand = []
    for x in kept:
        if x is None:
            hand.append(None)
            continue
        y = torch.zeros(4, T, *x.shape[3:], dtype=x.dtype, device=dev)
        for b, n in enumerate([300, 300, 250, 250]):
            y[b, :n] = x[0, prompt[b]].flatten(0, 1)[:n]
        hand.append(y)
    ln = [300, 300, 250, 250]
    for _, draft, mask, q, acc, path in steps:
        for b, a in enumerate(acc.tolist()):
            for j in range(a):
                for y, d in zip(hand, draft):
                    if y is not None:
                        y[b, ln[b] + j] = d[b, path[b][j]]
            ln[b] += a
    o, lse = A.attn_decode_splitkv(q1, hand[0], hand[1], ints(ln, dev), k_scale=hand[2], v_scale=hand[3],
                                   num_splits=1)
    o2, lse2 = A.attn_decode_paged(q1, after[0][0], after[1][0], got[-4], got[-3], num_splits=1,
                                   **(dict(k_scale=after[2][0], v_scale=after[3][0]) if coded else {}))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # captured: from the same start, the same end
    def restore():
        for x, y in zip(pool, kept):
            if x is not None:
                x.copy_(y)
    restore()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs = run()
    for _ in range(2):
        restore()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, got, strict=True))
        assert all(x is None or torch.equal(x, y) for x, y in zip(pool, after))
    del contig
    device_clean()


def test_calls_on_other_streams_do_not_meet(cuda_device):
    """Two forks at once, each with its own workspace, on streams of their own."""
    dev = cuda_device
    jobs = []
    for s in range(2):
        r = random.Random(s)
        lens, table, refs, width, N = random_pool(r, 30, 128, 900, 100)
        caches = make_cache("bf16", (2, N, 128), 2, s, dev)
        parents, keep, new = random_children(r, lens, 30, 128, width)
        want = as_bytes(caches)
        res = OP.fork(want, table, lens, refs, parents, keep, new, 128, width)
        a = (pad(table, width, dev), ints(lens, dev), ints(refs, dev), ints(parents, dev))
        jobs.append((caches, a, dict(keep_lens=ints(keep, dev), new_lens=ints(new, dev)), want, res))
    torch.cuda.synchronize()
    got = [A.attn_pages_fork(c[0], c[1], *a, **kw, stream=torch.cuda.Stream()) for c, a, kw, _, _ in jobs]
    torch.cuda.synchronize()
    for (c, _, _, want, res), x in zip(jobs, got):
        assert same(c, want)
        if res[0] is not None:
            assert x[0].tolist() == res[0] and x[2].tolist() == res[2]
    device_clean()
