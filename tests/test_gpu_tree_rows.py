"""Tree decode over coded caches where single rows or tokens stand far out: a sink token over a long tail.

Tolerance, per element of o = sum_t w_t v_t with v_t = code_t * scale_t: the weight times its V scale is rounded once to
f16 (11 significant bits: half a step is at most 2^-11 of it), scores move a weight by at most 2^-11 (128 products
in fp32, |score| < 64), and the result is rounded to bf16 (2^-8).  f16's step stops shrinking 2^-14 below 1:
the kernel promises that the row's largest product w_t |scale_t| is held as 2^3 or more, so another is off by at most
2^-25 / 2^3 = 2^-28 of the largest where it is below 2^-17 of it.  The cases keep their tails
above that, or the scales of the sink's tile alike (the reference then lies 2^10 below the largest), so

    |o error| <= 2^-8 |o| + (2^-11 + 2^-11) sum_t w_t |v_t|,    |lse error| <= 2^-11 + 2^-20 |lse|.
"""
import functools
import math

import numpy as np
import pytest
import torch

from exact_long_context_tmem_b200 import attn as A
from tests.parity import device_clean, to_np

pytestmark = pytest.mark.gpu
CODED = ["fp8", "int8", "int4"]


def encode(x, kind):
    """Whole numbers of at most 7 as codes of a cache (all three kinds hold them exactly)."""
    if kind == "fp8":
        return x.float().to(torch.float8_e4m3fn).view(torch.uint8)
    if kind == "int8":
        return x.to(torch.int8)
    y = (x.to(torch.int32) & 15).to(torch.uint8)
    return y[..., 0::2] | (y[..., 1::2] << 4)


def sink_cache(T, n_q, G, level, k_ratio, v_shift, seed, where):
    """One sequence of T tokens: a tail whose scores are 0 (in units of log2) to within a tenth or so, and a sink
    `level` above it at slot `where`, its K scale k_ratio and its V scale 2^-v_shift of the others', its V of
    the other sign.  Returns q [n_q, G, D] and the codes and scales of K and V, [T, D] and [T]."""
    g = torch.Generator().manual_seed(seed)
    D = 128
    q0 = torch.randn(D, generator=g)
    q = (q0 + 0.02 * torch.randn(n_q, G, D, generator=g)).to(torch.bfloat16)
    kc = torch.randint(-1, 2, (T, D), generator=g) * (torch.rand(T, D, generator=g) < 0.02)
    vc = torch.randint(3, 8, (T, D), generator=g)
    ks = 0.97 + 0.03 * torch.rand(T, generator=g)
    vs = 0.97 + 0.03 * torch.rand(T, generator=g)
    kc[where] = (q0 * 3).round().clamp(-7, 7).to(kc.dtype)
    vc[where] = -vc[where]
    ks[where], vs[where] = 0.97 * k_ratio, 0.97 * 2.0**-v_shift
    dot = float(q0 @ kc[where].float())
    ks *= level / (dot * float(ks[where]) * math.log2(math.e) / math.sqrt(D))
    return q, kc, ks, vc, vs


def rows_in_float64(q, kc, ks, vc, vs, mask, n_q):
    """o, lse and sum w |v| of every draft and head over one sequence."""
    k, v = to_np(kc) * to_np(ks)[:, None], to_np(vc) * to_np(vs)[:, None]
    T, base = len(k), len(k) - n_q
    s = np.einsum("igd,td->igt", to_np(q), k) / math.sqrt(q.shape[-1])
    for i in range(n_q):
        for t in range(max(base, 0), T):
            if not (int(mask[i]) >> (t - base)) & 1:
                s[i, :, t] = -np.inf
    top = s.max(-1, keepdims=True)
    e = np.exp(s - np.maximum(top, -1e300))
    w = e / np.maximum(e.sum(-1, keepdims=True), 1e-300)
    return w @ v, (top + np.log(np.maximum(e.sum(-1, keepdims=True), 1e-300)))[..., 0], w @ np.abs(v)


def run_shared(kind, q, kc, ks, vc, vs, mask, dev):
    """As many sequences as processors, with one page table over one pool: a CTA walks a whole item."""
    T, D = kc.shape
    B = torch.cuda.get_device_properties(dev).multi_processor_count
    pages = -(-T // 128)
    pad = pages * 128 - T

    def pool(x):
        x = torch.cat([x, x.new_zeros(pad, *x.shape[1:])])
        return x.view(pages, 128, 1, *x.shape[1:]).contiguous().to(dev)
    table = torch.arange(pages, dtype=torch.int32, device=dev).repeat(B, 1)
    qb = q.to(dev).repeat(B, 1, 1, 1).contiguous()
    lens = torch.full((B,), T, dtype=torch.int32, device=dev)
    m = torch.tensor(mask, dtype=torch.int64, device=dev).repeat(B, 1)
    return A.attn_decode_tree_paged(qb, pool(encode(kc, kind)), pool(encode(vc, kind)), table, lens, m,
                                    k_scale=pool(ks), v_scale=pool(vs))


def check_rows(o, lse, ref):
    ro, rl, size = ref
    assert torch.isfinite(o.float()).all()
    worst = (np.abs(to_np(o) - ro) / (2.0**-8 * np.abs(ro) + 2.0**-10 * size)).max()  # every sequence is the same
    assert worst <= 1, f"o: {worst:.3f} of its tolerance"
    assert (np.abs(to_np(lse) - rl) <= 2.0**-11 + 2.0**-20 * np.abs(rl)).all()


@functools.lru_cache(maxsize=1)  # the three kinds hold the same values
def sink_case(T, n_q, level, k_ratio, v_shift, where):
    mask = [(1 << (i + 1)) - 1 for i in range(n_q)]
    c = sink_cache(T, n_q, 4, level, k_ratio, v_shift, 3, where)
    return c, mask, rows_in_float64(*c, mask, n_q)


@pytest.mark.parametrize("kind", CODED)
@pytest.mark.parametrize("n_q", [8, 40])
@pytest.mark.parametrize("T,level,k_ratio,v_shift,where", [(32768, 19, 0.85, 3, 0), (131072, 20, 0.85, 4, 0),
                                                           (131072, 20.5, 0.87, 4, 300), (131072, 21, 0.88, 4, 65000),
                                                           (131072, 21, 0.99, 6, 65000), (131072, 18, 1.0, 0, 5),
                                                           (100003, 19, 0.6, 0, 131)])
def test_a_sink_does_not_cost_the_tail(cuda_device, kind, n_q, T, level, k_ratio, v_shift, where):
    """The tail holds 6 to 35 % of the weight and nearly all of the output; one token far above it, whose scales are the
    smallest of its tile, sets the row's reference."""
    c, mask, ref = sink_case(T, n_q, level, k_ratio, v_shift, where)
    o, lse = run_shared(kind, *c, mask, cuda_device)
    check_rows(o, lse, ref)
    device_clean()


@pytest.mark.parametrize("kind", CODED)
@pytest.mark.parametrize("n_q", [8, 40])
@pytest.mark.parametrize("tail", [0.0, 2.0**-70])
def test_v_scales_of_next_to_nothing_over_a_long_cache(cuda_device, kind, n_q, tail):
    """V scales that are all zero (or nearly): the sum of weights is taken relative to a product that is not there."""
    T, mask = 131072, [(1 << (i + 1)) - 1 for i in range(n_q)]
    q, kc, ks, vc, vs = sink_cache(T, n_q, 4, 12, 1.0, 0, 4, 77)
    vs = vs * tail
    c = q, kc, ks, vc, vs
    o, lse = run_shared(kind, *c, mask, cuda_device)
    if tail == 0:
        assert (o == 0).all()
    check_rows(o, lse, [x + (1e-300 if i == 2 else 0) for i, x in enumerate(rows_in_float64(*c, mask, n_q))])
    device_clean()


@pytest.mark.parametrize("kind", CODED)
@pytest.mark.parametrize("n_q,G", [(7, 4), (40, 4), (9, 1)])
@pytest.mark.parametrize("big", [2.0**16, 2.0**40, 2.0**116])
def test_a_row_of_huge_queries_leaves_the_others_alone(cuda_device, kind, n_q, G, big):
    """Queries come as f16 relative to a power of two; a padded draft's may be anything (here of up to 2^116, whether
    it sees nothing or the prefix), and one head's far from another's.  A row's own elements span 2^29 of
    its largest exactly, so the ordinary rows keep the ordinary tolerance.  (The huge rows' own scores are
    beyond what fp32 differences can tell apart, 2^25, and their outputs are not looked at.)"""
    D, Hkv, dev = 128, 2, cuda_device
    g = torch.Generator().manual_seed(n_q)
    lens = [n_q, 700, 300]
    T = max(lens)
    kc, vc = (torch.randint(-7, 8, (3, T, Hkv, D), generator=g) for _ in range(2))
    ks, vs = (0.1 * (1 + torch.rand(3, T, Hkv, generator=g)) for _ in range(2))
    q = torch.randn(3, n_q, Hkv * G, D, generator=g).to(torch.bfloat16)
    mask = np.array([[(1 << (i + 1)) - 1 for i in range(n_q)]] * 3, dtype=np.int64)
    usual = torch.ones(3, n_q, Hkv * G, dtype=torch.bool)
    for b in (0, 1):
        for i in (2, n_q - 1):  # padding: sees no draft (in sequence 0, which is drafts alone, nothing)
            mask[b, i] = 0
            q[b, i] *= big
            usual[b, i] = False
    q[2, :, 0] *= big  # a head
    usual[2, :, 0] = False
    o, lse = A.attn_decode_tree(q.to(dev), encode(kc, kind).to(dev), encode(vc, kind).to(dev),
                                torch.tensor(lens, dtype=torch.int32, device=dev), torch.from_numpy(mask).to(dev),
                                k_scale=ks.to(dev), v_scale=vs.to(dev))
    for b, n in enumerate(lens):
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            ro, rl, size = rows_in_float64(q[b, :, heads], kc[b, :n, h], ks[b, :n, h], vc[b, :n, h], vs[b, :n, h],
                                           mask[b], n_q)
            u = usual[b, :, heads].numpy()
            err = np.abs(to_np(o[b, :, heads]) - ro) / (2.0**-8 * np.abs(ro) + 2.0**-10 * size + 1e-300)
            worst = err[u].max(initial=0.0)
            assert worst <= 1, f"o: {worst:.3f} of its tolerance"
            assert (np.abs(to_np(lse[b, :, heads])[u] - rl[u]) <= 2.0**-11 + 2.0**-20 * np.abs(rl[u])).all()
    assert (o[0, 2] == 0).all() and torch.isneginf(lse[0, 2]).all()
    device_clean()
