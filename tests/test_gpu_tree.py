"""GPU parity of the tree decode against the float64 definition (oracle/tree.py).

Tolerance, per element of o = sum_t w_t v_t with weights w = softmax: each weight (times its V scale for a
coded cache) is rounded once to bf16: 8 significant bits, so half a step is at most 2^-8 of it.  The fp32 arithmetic of scores, exponentials
and sums stays below 2^-16 of each term at these sizes (|score| < 64: its rounding, 128 products
in fp32, moves a weight by < 128 * 64 * 2^-24 = 2^-11 at the very worst and is charged as that),
and the result is rounded to bf16 (2^-8 of it).  So |error| <= 2^-8 |o| + (2^-8 + 2^-11) sum_t w_t |v_t|,
and |lse error| <= 2^-11 + 2^-20 |lse|.
"""
import math

import numpy as np
import pytest
import torch

from exact_long_context_tmem_b200 import attn as A
from exact_long_context_tmem_b200 import inputs as I
from oracle import fp8 as F8
from oracle import intq as IQ
from oracle import tree as OT
from tests.parity import device_clean, to_np

pytestmark = pytest.mark.gpu
KINDS = {"bf16": {}, "fp8": {"kv_fp8": True}, "int8": {"kv_bits": 8}, "int4": {"kv_bits": 4}}


def random_masks(g, B, n_q):
    """Trees in topological order: a draft sees itself and its ancestors."""
    out = np.zeros((B, n_q), dtype=np.uint64)
    for b in range(B):
        for i in range(n_q):
            p = int(g.integers(max(-1, i - 6), i))
            out[b, i] = np.uint64(1 << i) | (out[b, p] if p >= 0 else np.uint64(0))
    return torch.from_numpy(out.view(np.int64))


def make(kind, B, n_q, Hq, Hkv, lens, Tmax, D=128, seed=0):
    w = I.Workload("tree", "decode", B=B, Hq=Hq, Hkv=Hkv, D=D, seed=900 + seed, **KINDS[kind])
    d = I.decode_inputs(w, lens=torch.tensor(lens, dtype=torch.int32), Tmax=Tmax)
    g = torch.Generator().manual_seed(77 + seed)
    d["q"] = torch.randn(B, n_q, Hq, D, generator=g).to(torch.bfloat16)
    d["mask"] = random_masks(np.random.default_rng(seed), B, n_q)
    return d


def values(d, kind):
    if kind == "bf16":
        return to_np(d["k"]), to_np(d["v"]), None, None
    if kind == "fp8":
        kv = F8.e4m3_decode(d["k_codes"]), F8.e4m3_decode(d["v_codes"])
    else:
        kv = tuple(IQ.int_values(d[x], int(kind[3:])) for x in ("k_codes", "v_codes"))
    return kv + (d["k_scale"], d["v_scale"])


def caches(d, kind, dev):
    if kind == "bf16":
        return (d["k"].to(dev), d["v"].to(dev)), {}
    return (d["k_codes"].to(dev), d["v_codes"].to(dev)), dict(k_scale=d["k_scale"].to(dev),
                                                              v_scale=d["v_scale"].to(dev))


def small_products(d, kind):
    """max_t (w_t |v_scale_t|) * sum_t |code_t| over the slots each row sees, [B, n_q, Hq, D]."""
    k, v, ks, vs = values(d, kind)
    q, vs, ks = to_np(d["q"]), to_np(vs), to_np(ks)
    B, n_q, Hq, D = q.shape
    G = Hq // k.shape[2]
    out = np.zeros(q.shape)
    for b, n in enumerate(d["kv_lens"].tolist()):
        for i in range(n_q):
            m = int(d["mask"][b, i]) % 2**64
            see = [t for t in range(n) if t < n - n_q or (m >> (t - n + n_q)) & 1]
            for h in range(Hq):
                x = q[b, i, h] @ (k[b, see, h // G] * ks[b, see, h // G, None]).T / math.sqrt(D)
                w = np.exp(x - x.max())
                top = (w / w.sum() * np.abs(vs[b, see, h // G])).max()
                out[b, i, h] = top * np.abs(v[b, see, h // G]).sum(0)
    return out


def check(o, lse, d, kind, q_lens=None, mask=None, small=0.0):
    k, v, ks, vs = values(d, kind)
    mask = d["mask"] if mask is None else mask
    D = d["q"].shape[-1]
    kw = dict(scale=1 / math.sqrt(D), q_lens=q_lens, k_scale=ks)
    m = mask.numpy().view(np.uint64)
    ro, rl = OT.decode_tree(d["q"], k, v, d["kv_lens"], m, v_scale=vs, **kw)
    size, _ = OT.decode_tree(d["q"], k, np.abs(v), d["kv_lens"], m, v_scale=None if vs is None else vs.abs(), **kw)
    o, lse = to_np(o), to_np(lse)
    assert np.isfinite(o).all()
    err = np.abs(o - ro)
    worst = (err / (2.0**-8 * np.abs(ro) + (2.0**-8 + 2.0**-11) * size + small + 1e-30)).max(initial=0.0)
    assert worst <= 1, f"o: {worst:.3f} of its tolerance"
    np.testing.assert_array_equal(np.isneginf(lse), np.isneginf(rl))
    f = np.isfinite(rl)
    assert (np.abs(lse[f] - rl[f]) <= 2.0**-11 + 2.0**-20 * np.abs(rl[f])).all()
    return worst


def tree(d, kind, dev, q_lens=None, mask=None, **kw):
    (k, v), sc = caches(d, kind, dev)
    mask = d["mask"] if mask is None else mask
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32, device=dev)
    return A.attn_decode_tree(d["q"].to(dev), k, v, d["kv_lens"].to(dev), mask.to(dev), q_lens=ql, **sc, **kw)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("n_q,Hq,Hkv", [(1, 4, 2), (8, 32, 8), (33, 8, 2), (64, 8, 2), (17, 7, 1), (64, 32, 2),
                                        (5, 3, 3), (43, 3, 1)])
def test_matches_definition(cuda_device, kind, n_q, Hq, Hkv):
    lens = [n_q, 700, max(n_q, 129), 1024]
    d = make(kind, 4, n_q, Hq, Hkv, lens, 1024, seed=n_q)
    check(*tree(d, kind, cuda_device), d, kind)
    device_clean()


@pytest.mark.parametrize("n_q,Hq,Hkv", [(3, 8, 8), (20, 16, 2), (64, 12, 4), (40, 128, 1), (2, 71, 1)])
def test_head_dim_64_and_wide_groups(cuda_device, n_q, Hq, Hkv):
    d = make("bf16", 2, n_q, Hq, Hkv, [max(n_q, 200), 513], 600, D=64, seed=5)
    check(*tree(d, "bf16", cuda_device), d, "bf16")
    device_clean()


@pytest.mark.parametrize("kind", list(KINDS))
def test_uneven_drafts_and_rows_that_see_nothing(cuda_device, kind):
    n_q = 24
    lens, q_lens = [0, 24, 1, 300, 256, 130, 999, 17], [5, 24, 1, 0, 13, 3, 24, 17]
    d = make(kind, 8, n_q, 8, 2, lens, 1024, seed=3)
    mask = d["mask"].clone()
    mask[1, 0] = 0      # the whole sequence is drafts: this row sees nothing at all
    mask[1, 7] = 1 << 3  # sees another draft, not itself
    mask[4, :] = -1      # bits past q_lens are ignored
    mask[6, 2] = 0      # sees the prefix alone
    o, lse = tree(d, kind, cuda_device, q_lens=q_lens, mask=mask)
    check(o, lse, d, kind, q_lens=q_lens, mask=mask)
    assert torch.isneginf(lse[1, 0]).all() and (o[1, 0] == 0).all()
    for b, n in enumerate(q_lens):
        assert torch.isneginf(lse[b, n:]).all() and (o[b, n:] == 0).all()
    device_clean()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("page_size", [128, 384])
def test_paged_equals_contiguous(cuda_device, kind, page_size):
    n_q, lens, q_lens = 19, [900, 19, 385, 1152, 0], [19, 19, 4, 11, 19]
    d = make(kind, 5, n_q, 8, 2, lens, 1152, seed=8)
    pd = I.paged_inputs(d, page_size, seed=4)
    o, lse = tree(d, kind, cuda_device, q_lens=q_lens)
    (k, v), sc = caches(pd, kind, cuda_device)
    dev = cuda_device
    op, lp = A.attn_decode_tree_paged(d["q"].to(dev), k, v, pd["page_table"].to(dev), d["kv_lens"].to(dev),
                                      d["mask"].to(dev), q_lens=torch.tensor(q_lens, dtype=torch.int32, device=dev),
                                      **sc)
    assert torch.equal(o, op) and torch.equal(lse, lp)
    check(op, lp, d, kind, q_lens=q_lens)
    device_clean()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_chain_equals_multi_token_decode(cuda_device, kind):
    """A chain mask is attn_decode_multi's causal reading; both keep the same tolerance."""
    d = make(kind, 3, 4, 8, 2, [500, 4, 129], 512, seed=6)
    chain = torch.tensor([[(1 << (i + 1)) - 1 for i in range(4)]] * 3, dtype=torch.int64)
    o, lse = tree(d, kind, cuda_device, mask=chain)
    check(o, lse, d, kind, mask=chain)
    (k, v), sc = caches(d, kind, cuda_device)
    om, lm = A.attn_decode_multi(d["q"].to(cuda_device), k, v, d["kv_lens"].to(cuda_device), **sc)
    check(om, lm, d, kind, mask=chain)
    device_clean()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("n_q", [6, 48])
def test_nonfinite_drafts_reach_only_the_rows_that_see_them(cuda_device, kind, n_q):
    """Drafts hold NaN or infinities in V (by the scale for INT8): rows that see none of them are as if
    they were not there, rows that see one get it."""
    dev = cuda_device
    d = make(kind, 3, n_q, 8, 2, [n_q, 127 + n_q // 2, 640], 640, seed=2)
    bad = [2, 5]
    clean = {x: y.clone() if isinstance(y, torch.Tensor) else y for x, y in d.items()}
    for b in range(3):
        for j in bad:
            t = int(d["kv_lens"][b]) - n_q + j
            if kind == "bf16":
                d["v"][b, t, 0, 3] = math.inf if j == 2 else math.nan
            elif kind == "fp8":
                d["v_codes"][b, t, 0, 3] = 0x7F
            else:
                d["v_scale"][b, t, 0] = math.nan
    o, lse = tree(d, kind, dev)
    oc, lc = tree(clean, kind, dev)
    seen = (d["mask"] & sum(1 << j for j in bad)) != 0
    assert seen.any() and not seen.all()
    G = 4
    hit = torch.zeros(o.shape, dtype=torch.bool)
    cols = slice(None) if kind == "int8" else slice(3, 4)
    for b, i in seen.nonzero().tolist():
        hit[b, i, :G, cols] = True
    bad_out = ~torch.isfinite(o.float().cpu())
    assert torch.equal(bad_out, hit)
    keep = (~seen).to(dev)
    assert torch.equal(o[keep], oc[keep]) and torch.equal(lse[keep], lc[keep])
    # Rows that see one: V (and its scale, relative to which a coded cache's weights are taken) has no part in the
    # lse, so both calls are within the lse tolerance of one value, and within twice that of each other.
    assert ((lse - lc).abs() <= 2 * (2.0**-11 + 2.0**-20 * lc.abs())).all()
    if kind == "bf16":
        only_inf = ((d["mask"] & (1 << 2)) != 0) & ((d["mask"] & (1 << 5)) == 0)
        for b, i in only_inf.nonzero().tolist():
            assert torch.isposinf(o[b, i, :G, 3].float()).all()
    device_clean()


@pytest.mark.parametrize("kind", list(KINDS))
def test_unseen_slots_may_hold_anything(cuda_device, kind):
    """A draft that nobody sees, and slots past the length, hold NaN in K and V (NaN scales for coded)."""
    n_q = 9
    d = make(kind, 2, n_q, 8, 2, [140, 9], 256, seed=12)
    mask = d["mask"] & ~(1 << 4)
    want = tree(d, kind, cuda_device, mask=mask)
    for b, n in enumerate([140, 9]):
        for t in [n - n_q + 4] + list(range(n, 256)):
            if kind == "bf16":
                d["k"][b, t] = d["v"][b, t] = math.nan
            else:
                d["k_scale"][b, t] = d["v_scale"][b, t] = math.nan
                if kind == "fp8":
                    d["k_codes"][b, t] = d["v_codes"][b, t] = 0x7F
    got = tree(d, kind, cuda_device, mask=mask)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    device_clean()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("n_q,G", [(4, 4), (40, 4)])
def test_many_sequences_share_ctas(cuda_device, kind, n_q, G):
    """More (sequence, head) items than CTAs, so ranges begin and end inside items; and repeats are exact."""
    g = np.random.default_rng(4)
    lens = g.integers(n_q, 900, size=60).tolist()
    lens[7], lens[31] = 0, n_q
    d = make(kind, 60, n_q, 4 * G, 4, lens, 900, seed=14)
    o, lse = tree(d, kind, cuda_device)
    for _ in range(3):
        o2, l2 = tree(d, kind, cuda_device)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    # the definition on a sample of the sequences
    pick = [0, 7, 31, 59]
    sub = {x: (y[pick] if isinstance(y, torch.Tensor) else y) for x, y in d.items()}
    check(o[pick], lse[pick], sub, kind)
    device_clean()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("n_q,G", [(40, 4), (64, 4), (60, 7), (16, 4), (17, 4), (21, 3), (64, 1), (1, 64), (1, 65)])
def test_uneven_drafts_around_a_row_slot(cuda_device, kind, n_q, G):
    """Sequences whose drafts fill one slot of rows, a part of it or more, one behind the other on a CTA."""
    g = np.random.default_rng(n_q)
    tps, B = min(128 // G, 64), 48
    q_lens = [min(n_q, max(0, int(x))) for x in g.choice([0, 1, tps // 2, tps - 1, tps, tps + 1, 2 * tps, n_q], B)]
    lens = [max(q, int(x)) for q, x in zip(q_lens, g.integers(1, 700, size=B))]
    d = make(kind, B, n_q, 4 * G, 4, lens, 704, seed=n_q + G)
    o, lse = tree(d, kind, cuda_device, q_lens=q_lens)
    again = tree(d, kind, cuda_device, q_lens=q_lens)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    pick = [0, 1, 2, 3, 20, 21, 46, 47]
    sub = {x: (y[pick] if isinstance(y, torch.Tensor) else y) for x, y in d.items()}
    check(o[pick], lse[pick], sub, kind, q_lens=[q_lens[b] for b in pick])
    for b, n in enumerate(q_lens):
        assert torch.isneginf(lse[b, n:]).all() and (o[b, n:] == 0).all()
    device_clean()


def test_bad_page_is_reported_and_stays_local(cuda_device):
    dev = cuda_device
    d = make("bf16", 2, 5, 8, 2, [500, 300], 512, seed=1)
    pd = I.paged_inputs(d, 128, seed=4)
    (k, v), _ = caches(pd, "bf16", dev)
    args = (d["kv_lens"].to(dev), d["mask"].to(dev))
    want, _ = A.attn_decode_tree_paged(d["q"].to(dev), k, v, pd["page_table"].to(dev), *args)
    table = pd["page_table"].clone()
    table[0, 1] = pd["num_pages"] + 3
    got, _ = A.attn_decode_tree_paged(d["q"].to(dev), k, v, table.to(dev), *args)
    assert torch.equal(want[1], got[1]) and torch.isfinite(got.float()).all()
    st, site = A.attn_device_status(reset=True)
    assert (st, site) == (A.ATTN_ERR_INVALID_ARG, 60)
    device_clean()


def test_captured_call_replays_with_new_lengths(cuda_device):
    dev, n_q = cuda_device, 12
    d = make("bf16", 3, n_q, 8, 2, [600, 12, 333], 640, seed=20)
    (k, v), _ = caches(d, "bf16", dev)
    q, lens, mask = d["q"].to(dev), d["kv_lens"].to(dev), d["mask"].to(dev)
    q_lens = torch.full((3,), n_q, dtype=torch.int32, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        A.attn_decode_tree(q, k, v, lens, mask, q_lens=q_lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = A.attn_decode_tree(q, k, v, lens, mask, q_lens=q_lens)
    for new in ([600, 12, 333], [12, 640, 0], [129, 300, 640]):
        nl = [min(n_q, x) for x in new]
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        q_lens.copy_(torch.tensor(nl, dtype=torch.int32))
        k2 = torch.randn(k.shape, device=dev).to(torch.bfloat16)
        k.copy_(k2)
        v.copy_(k2.flip(1))
        g.replay()
        d2 = dict(d, k=k.cpu(), v=v.cpu(), kv_lens=lens.cpu())
        check(o, lse, d2, "bf16", q_lens=nl)
    device_clean()


def test_two_streams_at_once(cuda_device):
    dev = cuda_device
    ds = [make("fp8", 4, 16, 16, 4, [2000, 1500, 16, 900], 2048, seed=s) for s in (1, 2)]
    want = [tree(d, "fp8", dev) for d in ds]
    dev_in = []
    for d in ds:
        (k, v), sc = caches(d, "fp8", dev)
        dev_in.append(((d["q"].to(dev), k, v, d["kv_lens"].to(dev), d["mask"].to(dev)), sc))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    for _ in range(5):
        got = [A.attn_decode_tree(*a, **sc, stream=s) for (a, sc), s in zip(dev_in, streams)]
        torch.cuda.synchronize()
        for w, x in zip(want, got):
            assert torch.equal(w[0], x[0]) and torch.equal(w[1], x[1])
    device_clean()


def test_empty_calls(cuda_device):
    dev = cuda_device
    k = torch.zeros(2, 0, 2, 128, dtype=torch.bfloat16, device=dev)
    q = torch.ones(2, 3, 4, 128, dtype=torch.bfloat16, device=dev)
    lens = torch.zeros(2, dtype=torch.int32, device=dev)
    mask = torch.full((2, 3), 7, dtype=torch.int64, device=dev)
    o, lse = A.attn_decode_tree(q, k, k, lens, mask)
    assert (o == 0).all() and torch.isneginf(lse).all()
    o, lse = A.attn_decode_tree(q[:, :0], k, k, lens, mask[:, :0])
    assert o.shape == (2, 0, 4, 128) and lse.shape == (2, 0, 4)
    device_clean()


@pytest.mark.parametrize("kind", ["fp8", "int8", "int4"])
@pytest.mark.parametrize("n_q", [7, 40])
@pytest.mark.parametrize("how", ["wide", "zeros", "negative", "one huge draft", "steep"])
def test_scales_of_any_range(cuda_device, kind, n_q, how):
    """V scales over 2^40, zero and negative scales, a draft whose scales are 2^60 of the others', K scales over 2^6
    (scores up to 60 or so).  A coded cache's weights times V scales are f16 numbers relative to (at least
    2^-8 of) the row's largest such product p: below f16's normal range they are off by up to 2^-25, 2^-17 of
    p, each, which adds 2^-17 p sum_t |code_t| to the tolerance.  That matters where the scales differ by
    2^40: then an element of o may owe its whole size to products far below p."""
    g = torch.Generator().manual_seed(5)
    d = make(kind, 3, n_q, 8, 2, [600, n_q, 333], 600, seed=4)
    if how == "wide":
        d["v_scale"] *= 2.0 ** torch.randint(-20, 21, d["v_scale"].shape, generator=g)
    elif how == "zeros":
        d["v_scale"] *= torch.randint(0, 2, d["v_scale"].shape, generator=g)
        d["k_scale"] *= torch.randint(0, 2, d["k_scale"].shape, generator=g)
    elif how == "negative":
        d["v_scale"] *= torch.randint(0, 2, d["v_scale"].shape, generator=g) * 2 - 1
        d["k_scale"] *= torch.randint(0, 2, d["k_scale"].shape, generator=g) * 2 - 1
    elif how == "steep":
        d["k_scale"] *= 2.0 ** torch.randint(-3, 4, d["k_scale"].shape, generator=g)
    else:
        for b, n in enumerate([600, n_q, 333]):
            d["v_scale"][b, n - n_q + 2] *= 2.0**60
    check(*tree(d, kind, cuda_device), d, kind, small=2.0**-17 * small_products(d, kind))
    device_clean()


@pytest.mark.parametrize("kind", list(KINDS))
def test_queries_of_any_size(cuda_device, kind):
    """Queries times 2^60 with K scales (bf16: K) over 2^60, and a sequence whose queries are all zero."""
    d = make(kind, 2, 9, 8, 2, [300, 200], 300, seed=9)
    d["q"] *= 2.0**60
    d["q"][1] = 0
    if kind == "bf16":
        d["k"] *= 2.0**-60
    else:
        d["k_scale"] *= 2.0**-60
    check(*tree(d, kind, cuda_device), d, kind)
    device_clean()


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_more_drafts_than_tokens(cuda_device, kind):
    """A length below the number of drafts: the cache holds the last of them only."""
    q_lens = [9, 9, 9]
    d = make(kind, 3, 9, 4, 2, [3, 1, 8], 128, seed=31)
    mask = torch.full((3, 9), -1, dtype=torch.int64)
    mask[0, 2] = (1 << 6) - 1  # none of the three that are there
    o, lse = tree(d, kind, cuda_device, q_lens=q_lens, mask=mask)
    check(o, lse, d, kind, q_lens=q_lens, mask=mask)
    assert torch.isneginf(lse[0, 2]).all()
    device_clean()


def test_outputs_and_workspace_of_the_caller(cuda_device):
    dev = cuda_device
    d = make("fp8", 2, 20, 16, 4, [700, 333], 768, seed=40)
    (k, v), sc = caches(d, "fp8", dev)
    args = (d["q"].to(dev), k, v, d["kv_lens"].to(dev), d["mask"].to(dev))
    want, wl = A.attn_decode_tree(*args, **sc)
    need = A.attn_decode_tree_workspace_bytes(2, 16, 4, 128, 768, 20)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    o = torch.full_like(want, math.nan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, none = A.attn_decode_tree(*args, **sc, o=o, ws=ws, want_lse=False, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert got is o and none is None and torch.equal(o, want)
    lse = torch.empty_like(wl)
    A.attn_decode_tree(*args, **sc, o=o, lse=lse, ws=ws)
    assert torch.equal(lse, wl)
    with pytest.raises(A.AttnError):
        A.attn_decode_tree(*args, **sc, ws=ws[:-16])
    with pytest.raises(ValueError):
        A.attn_decode_tree(*args[:4], d["mask"].to(dev).int(), **sc)
    with pytest.raises(ValueError):
        A.attn_decode_tree(*args, **sc, q_lens=torch.ones(2, dtype=torch.int64, device=dev))
    device_clean()


def test_long_cache_past_32_bit_offsets(cuda_device):
    """One sequence of more than 2^31 elements of K: the last tiles are read where they are."""
    dev, T, n_q = cuda_device, 2**21 + 200, 5
    k = torch.zeros(1, T, 8, 128, dtype=torch.bfloat16, device=dev)
    v = torch.zeros_like(k)
    g = torch.Generator().manual_seed(3)
    k[0, -300:] = 3 * torch.randn(300, 8, 128, generator=g).to(torch.bfloat16).to(dev)
    v[0, -300:] = torch.randn(300, 8, 128, generator=g).to(torch.bfloat16).to(dev)
    q = (4 * torch.randn(1, n_q, 16, 128, generator=g)).to(torch.bfloat16)
    mask = random_masks(np.random.default_rng(5), 1, n_q)
    lens = torch.tensor([T], dtype=torch.int32)
    o, lse = A.attn_decode_tree(q.to(dev), k, v, lens.to(dev), mask.to(dev))
    # by hand: the zero keys have score 0 and value 0, so they only add their number to each sum
    kt, vt = to_np(k[0, -300:]), to_np(v[0, -300:])
    m = mask.numpy().view(np.uint64)[0]
    for i in range(n_q):
        see = np.array([t < 300 - n_q or bool(int(m[i]) >> (t - 300 + n_q) & 1) for t in range(300)])
        for h in range(16):
            s = to_np(q)[0, i, h] @ kt[see, h // 2].T / math.sqrt(128)
            total = np.exp(s).sum() + (T - 300)
            ref = np.exp(s) @ vt[see, h // 2] / total
            size = np.exp(s) @ np.abs(vt[see, h // 2]) / total
            assert (np.abs(to_np(o)[0, i, h] - ref) <= 2.0**-8 * np.abs(ref) + (2.0**-8 + 2.0**-11) * size).all()
            assert abs(float(lse[0, i, h]) - math.log(total)) <= 2.0**-11 + 2.0**-20 * math.log(total)
    device_clean()
