"""Operators of speculative and beam decoding over the KV cache: the measured cases.

Two groups that a serving loop uses together.  One verifies a tree of drafted tokens
against a contiguous or paged cache (bf16, FP8 E4M3, INT8 or INT4 codes) and then keeps the
accepted path: `attn_decode_tree`, `attn_decode_tree_paged`, `attn_tree_accept`.  The other
keeps the pages of a paged cache: copying pages, forking / truncating / growing / freeing
sequences over shared pages, and compacting the pool: `attn_pages_copy`, `attn_pages_fork`,
`attn_pages_compact`.

Each case names its operator in "op".  `run` computes it in elementary torch operations
where `own` is false and through the package's public calls where it is true.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # Verification of a short draft in one chat session: one small sequence, where the time is launches
        # and latency, not bytes.
        dict(name="tree_b1_n8_t2048_bf16", op="tree", kv="bf16", paged=False, page=128, B=1, Hq=32, Hkv=8, D=128,
             n_q=8, T=2048, ragged=False, uneven=False),
        # The long-context decode workload (batch 4, lengths 64K-128K, bf16) verifying 64 drafted tokens.
        dict(name="tree_b4_n64_t131072_bf16", op="tree", kv="bf16", paged=False, page=128, B=4, Hq=32, Hkv=8, D=128,
             n_q=64, T=131072, ragged=True, uneven=False),
        # The FP8 serving workload (batch 16, 32768 tokens, 512-token pages) verifying 16 drafted tokens.
        dict(name="tree_b16_n16_t32768_fp8", op="tree", kv="fp8", paged=True, page=512, B=16, Hq=32, Hkv=8, D=128,
             n_q=16, T=32768, ragged=False, uneven=False),
        # Odd sizes: groups of 7 query heads, up to 25 drafted tokens, ragged lengths in an INT8 pool of short pages.
        dict(name="tree_b8_n25_g7_t10007_int8", op="tree", kv="int8", paged=True, page=128, B=8, Hq=28, Hkv=4, D=128,
             n_q=25, T=10007, ragged=True, uneven=True),
        # Keeping the accepted path of 4 short drafts in two layers of a contiguous cache: latency.
        dict(name="accept_b4_n16_l2_bf16", op="accept", kv="bf16", paged=False, page=128, B=4, Hkv=8, D=128, n_q=16,
             T=1024, L=2),
        # A full batch of large trees, 16 layers of an FP8 pool.
        dict(name="accept_b64_n64_l16_fp8", op="accept", kv="fp8", paged=True, page=512, B=64, Hkv=8, D=128, n_q=64,
             T=700, L=16),
        # Copying a few pages of one layer (copy on write of single pages).
        dict(name="copy_n5_l1_bf16", op="copy", kv="bf16", page=128, Hkv=8, D=128, L=1, pages=64, n=5),
        # Duplicating many pages over eight layers (moving sequences inside a pool).
        dict(name="copy_n255_l8_bf16", op="copy", kv="bf16", page=128, Hkv=8, D=128, L=8, pages=600, n=255),
        # One beam step: 2 prompts x 4 beams, beams replaced by copies of better ones, each one token longer.
        dict(name="fork_b8_t2048_l4_bf16", op="fork", kv="bf16", page=128, Hkv=8, D=128, L=4, B=8, T=2048,
             pages=160, style="beam"),
        # A continuous-batching step over 256 sequences: forks, truncations after rejected drafts, growth,
        # finished sequences freed and new ones admitted.
        dict(name="fork_b256_t8192_l2_fp8", op="fork", kv="fp8", page=128, Hkv=2, D=128, L=2, B=256, T=8192,
             pages=16384, style="mixed"),
        # Compacting a small pool.
        dict(name="compact_p96_l2_bf16", op="compact", kv="bf16", page=128, Hkv=8, D=128, L=2, B=4, T=2048, pages=96),
        # Compacting a large, half-empty INT8 pool after many sequences have ended.
        dict(name="compact_p4096_l2_int8", op="compact", kv="int8", page=128, Hkv=8, D=128, L=2, B=64, T=8000,
             pages=4096),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "accept", "copy", "fork", "compact"])
    kv = rng.choice(["bf16", "fp8", "int8", "int4"])
    if op == "tree":
        D = rng.choice([64, 128]) if kv == "bf16" else 128
        while True:
            G, Hkv = rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([1, 2, 4, 8])
            n_q, B, T = _logint(rng, 1, 64), _logint(rng, 1, 48), _logint(rng, 16, 131072)
            # no more work or memory than the largest listed case
            if B * T <= 4 * 131072 and B * T * Hkv <= 4 * 131072 * 8 and B * T * G * Hkv * n_q <= 4 * 131072 * 32 * 48:
                break
        return dict(op="tree", kv=kv, paged=rng.random() < 0.5, page=rng.choice([128, 256, 384, 512]), B=B, Hq=G * Hkv,
                    Hkv=Hkv, D=D, n_q=n_q, T=max(T, n_q), ragged=rng.random() < 0.7,
                    uneven=rng.random() < 0.5)
    Hkv = rng.choice([1, 2, 4, 5, 8])
    D = rng.choice([64, 128]) if kv == "bf16" else 128
    page = rng.choice([128, 256, 512])
    if op == "accept":
        return dict(op="accept", kv=kv, paged=rng.random() < 0.5, page=page, B=_logint(rng, 1, 64), Hkv=Hkv, D=D,
                    n_q=_logint(rng, 2, 64), T=rng.randint(70, 900), L=_logint(rng, 1, 8))
    if op == "copy":
        pages = _logint(rng, 8, 300)
        return dict(op="copy", kv=kv, page=page, Hkv=Hkv, D=D, L=_logint(rng, 1, 6), pages=pages,
                    n=rng.randint(1, pages // 2))
    if op == "fork":
        B, T = _logint(rng, 1, 128), _logint(rng, 100, 4000)
        per = T // page + 2
        return dict(op="fork", kv=kv, page=page, Hkv=rng.choice([1, 2]), D=D, L=_logint(rng, 1, 4), B=B, T=T,
                    pages=2 * B * per + rng.randint(0, 37), style=rng.choice(["beam", "mixed"]))
    B, T = _logint(rng, 1, 64), _logint(rng, 100, 3000)
    return dict(op="compact", kv=kv, page=page, Hkv=rng.choice([1, 2, 4]), D=D, L=_logint(rng, 1, 3), B=B, T=T,
                pages=B * (T // page + 1) * 2 + rng.randint(1, 29))


# ------------------------------------------------------------------------------------ inputs

def _shape_rng(case):
    """Lengths, tables and page lists that only the case decides (so that `work` knows them)."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


ROW = {"bf16": 2.0, "fp8": 1.0, "int8": 1.0, "int4": 0.5}


def _cache(kv, lead, Hkv, D, g):
    """Cache tensors [*lead, Hkv, D]: N(0,1) values, coded caches with a scale per (token, KV head)."""
    if kv == "bf16":
        x = torch.empty(*lead, Hkv, D, device=DEV, dtype=torch.bfloat16)
        return x.normal_(generator=g), None
    n = math.prod(lead)
    row = D // 2 if kv == "int4" else D
    codes = torch.empty(n, Hkv, row, device=DEV, dtype=torch.int8 if kv == "int8" else torch.uint8)
    scale = torch.empty(n, Hkv, device=DEV)
    step = 1 << 17
    for i in range(0, n, step):
        x = torch.randn(min(step, n - i), Hkv, D, device=DEV, generator=g)
        top = x.abs().amax(-1)
        s = top / {"fp8": 448.0, "int8": 127.0, "int4": 7.0}[kv]
        scale[i:i + step] = s
        y = x / s[..., None]
        if kv == "fp8":
            codes[i:i + step] = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        elif kv == "int8":
            codes[i:i + step] = y.round().clamp(-127, 127).to(torch.int8)
        else:
            c = (y.round().clamp(-7, 7).to(torch.int32) & 15).to(torch.uint8)
            codes[i:i + step] = c[..., 0::2] | (c[..., 1::2] << 4)
    return codes.view(*lead, Hkv, row), scale.view(*lead, Hkv)


def _tree_lens(case):
    r = _shape_rng(case)
    B, T, n_q = case["B"], case["T"], case["n_q"]
    lens = [r.randint(max(n_q, T // 2), T) if case["ragged"] else T for _ in range(B)]
    q_lens = [r.randint(1, n_q) if case["uneven"] else n_q for _ in range(B)]
    return lens, q_lens


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _pool_lists(case):
    """Sequences over a pool: lengths, page tables (random pool order, shared prefixes) and reference counts."""
    r = _shape_rng(case)
    B, T, page, N = case["B"], case["T"], case["page"], case["pages"]
    order = list(range(N))
    r.shuffle(order)
    lens, table, refs = [], [], [0] * N
    width = T // page + 2
    for b in range(B):
        n = r.randint(max(1, T // 2), T)
        held = -(-n // page)
        shared = []
        if table and r.random() < 0.5:  # a common prompt: whole pages of an earlier sequence
            o = r.randrange(b)
            shared = table[o][:r.randint(0, min(lens[o] // page, (n - 1) // page))]
        pages = shared + [order.pop() for _ in range(held - len(shared))]
        for p in pages:
            refs[p] += 1
        lens.append(n)
        table.append(pages)
    return r, lens, table, refs, width


def _fork_lists(case):
    r, lens, table, refs, width = _pool_lists(case)
    B, page = case["B"], case["page"]
    if case["style"] == "beam":  # groups of 4 beams: each goes on from one of its group, one token longer
        parents = [min(B - 1, b - b % 4 + r.randrange(4)) for b in range(B)]
        keep = [lens[p] for p in parents]
        new = [k + 1 for k in keep]
    else:
        parents, keep, new = [], [], []
        for b in range(B):
            what = r.random()
            if what < 0.1:  # finished, nothing takes its place
                parents.append(-1), keep.append(0), new.append(0)
            elif what < 0.2:  # finished, a new prompt is admitted
                parents.append(-1), keep.append(0), new.append(r.randint(1, case["T"]))
            else:  # goes on (or forks another): rejected drafts cut off, room for the next ones
                p = b if what < 0.8 else r.randrange(B)
                k = max(0, lens[p] - r.randint(0, 40))
                parents.append(p), keep.append(k), new.append(k + r.randint(0, 64))
    held = [-(-n // page) for n in new]
    width = max([width] + held)
    return lens, table, refs, parents, keep, new, width


def _table(rows, width):
    return _ints([x + [-1] * (width - len(x)) for x in rows])


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    r = random.Random(seed)
    s = dict(case=case, op=op)
    if op == "tree":
        B, n, Hkv, D, T, page = case["B"], case["n_q"], case["Hkv"], case["D"], case["T"], case["page"]
        lens, q_lens = _tree_lens(case)
        s["q"] = torch.empty(B, n, case["Hq"], D, device=DEV, dtype=torch.bfloat16).normal_(generator=g)
        if case["paged"]:
            per = -(-T // page)
            order = list(range(B * per + 3))
            r.shuffle(order)
            s["table"] = _ints([order[b * per:(b + 1) * per] for b in range(B)])
            lead = (B * per + 3, page)
        else:
            s["table"] = None
            lead = (B, T)
        s["k"], s["ks"] = _cache(case["kv"], lead, Hkv, D, g)
        s["v"], s["vs"] = _cache(case["kv"], lead, Hkv, D, g)
        s["lens"], s["q_lens"] = _ints(lens), _ints(q_lens)
        masks = []
        for b in range(B):  # a tree in topological order: each token sees itself and its ancestors
            row = []
            for i in range(n):
                p = r.randint(max(-1, i - 6), i - 1)
                row.append((row[p] if p >= 0 else 0) | (1 << i))
            masks.append([m - (1 << 64) if m >> 63 else m for m in row])
        s["mask"] = torch.tensor(masks, dtype=torch.int64, device=DEV)
        return s
    Hkv, D, page, L = case["Hkv"], case["D"], case["page"], case["L"]
    if op == "accept":
        B, n, T = case["B"], case["n_q"], case["T"]
        sr = _shape_rng(case)
        acc, lens = _accept_lists(case, sr)
        per = -(-T // page)
        if case["paged"]:
            order = list(range(B * per + 1))
            r.shuffle(order)
            s["table"] = _ints([order[b * per:(b + 1) * per] for b in range(B)])
            lead = (L, B * per + 1, page)
        else:
            s["table"] = None
            lead = (L, B, T)
        s["lens"] = _ints(lens)
        s["n_acc"] = _ints([len(a) for a in acc])
        s["path"] = _ints([a + [0] * (n - len(a)) for a in acc])
    else:
        lead = (L, case["pages"], page)
        if op == "copy":
            order = list(range(case["pages"]))
            r.shuffle(order)
            s["src"], s["dst"] = _ints(order[:case["n"]]), _ints(order[case["n"]:2 * case["n"]])
        elif op == "fork":
            lens, table, refs, parents, keep, new, width = _fork_lists(case)
            s.update(table=_table(table, width), lens=_ints(lens), refs=_ints(refs), parents=_ints(parents),
                     keep=_ints(keep), new=_ints(new))
        else:
            _, lens, table, refs, width = _pool_lists(case)
            s.update(table=_table(table, width), refs=_ints(refs))
    s["k"], s["ks"] = _cache(case["kv"], lead, Hkv, D, g)
    s["v"], s["vs"] = _cache(case["kv"], lead, Hkv, D, g)
    return s


def _accept_lists(case, r):
    """Accepted paths.  The first steps often follow the first branch (tokens 0, 1, ...); the later ones lie
    past the kept prefix, so that running the same state again reads the same rows."""
    acc, lens = [], []
    for _ in range(case["B"]):
        n = case["n_q"]
        a = min(n, r.choice([0, 1, 2, 3, 4, 5, 6, 8]))
        first = r.randint(0, a)
        rest = list(range(a, n))
        more = min(a - first, len(rest))
        acc.append(list(range(first)) + sorted(r.sample(rest, more)))
        lens.append(r.randint(max(n, case["T"] // 2), case["T"]))
    return acc, lens


# ------------------------------------------------------------------------------------ plain forms

def _values(codes, scale, kv):
    """float32 values of a cache."""
    if kv == "bf16":
        return codes.float()
    if kv == "fp8":
        return codes.view(torch.float8_e4m3fn).float() * scale[..., None]
    if kv == "int8":
        return codes.float() * scale[..., None]
    x = codes.to(torch.int32)
    pair = torch.stack([x & 15, x >> 4], -1)
    return (pair - 16 * (pair > 7)).float().flatten(-2) * scale[..., None]


def _gathered(x, table):
    """[B, tokens, ...] view of a pool through its page table."""
    return x if x is None or table is None else x[table.long()].flatten(1, 2)


def _plain_tree(s):
    case = s["case"]
    B, n, Hq, Hkv, D = case["B"], case["n_q"], case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    k = _values(_gathered(s["k"], s["table"]), _gathered(s["ks"], s["table"]), case["kv"]).permute(0, 2, 3, 1)
    t = torch.arange(k.shape[-1], device=DEV)
    base = (s["lens"] - s["q_lens"])[:, None, None]
    rel = t - base  # index among the drafted tokens
    bit = (s["mask"][:, :, None] >> rel.clamp(0, 63)) & 1
    seen = (rel < 0) | ((rel < s["q_lens"][:, None, None]) & (bit == 1))
    seen &= (torch.arange(n, device=DEV) < s["q_lens"][:, None])[:, :, None]
    q = s["q"].float().view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    x = (q @ k).mul_(1.0 / math.sqrt(D)).view(B, Hkv, n, G, -1)
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = x.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    total = e.sum(-1, keepdim=True)
    v = _values(_gathered(s["v"], s["table"]), _gathered(s["vs"], s["table"]), case["kv"]).permute(0, 2, 1, 3)
    o = (e.view(B, Hkv, n * G, -1) @ v).view(B, Hkv, n, G, D) / total.masked_fill(total == 0, 1.0)
    lse = (m + total.log()).squeeze(-1)
    return (o.permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D).to(torch.bfloat16),
            lse.permute(0, 2, 1, 3).reshape(B, n, Hq))


def _caches(s):
    return [x for x in (s["k"], s["v"], s["ks"], s["vs"]) if x is not None]


def _plain_accept(s):
    page = s["k"].shape[2]
    table = s["table"]
    if table is None:
        table = torch.arange(s["case"]["B"], device=DEV)[:, None]
    j = torch.arange(s["path"].shape[1], device=DEV)
    base = (s["lens"] - s["case"]["n_q"]).long()
    b, step = (j < s["n_acc"][:, None]).nonzero(as_tuple=True)
    src = base[b] + s["path"].long()[b, step]
    dst = base[b] + step
    src = table[b, src // page].long() * page + src % page
    dst = table[b, dst // page].long() * page + dst % page
    for x in _caches(s):
        flat = x.flatten(1, 2)
        flat[:, dst] = flat[:, src]
    return s["k"], s["v"], s["ks"], s["vs"], (base + s["n_acc"]).int()


def _plain_copy(s):
    for x in _caches(s):
        x[:, s["dst"].long()] = x[:, s["src"].long()]
    return s["k"], s["v"], s["ks"], s["vs"]


def _plain_fork(s):
    page, N = s["case"]["page"], s["case"]["pages"]
    table, lens, refs = s["table"].long(), s["lens"].long(), s["refs"].long()
    parents = s["parents"].long()
    B, M = parents.numel(), table.shape[1]
    at = torch.arange(M, device=DEV)
    child = torch.arange(B, device=DEV)
    old = lens[parents.clamp(min=0)] * (parents >= 0)
    keep = torch.minimum(torch.minimum(s["keep"].long(), old), s["new"].long())
    full = keep // page
    cut = keep % page > 0
    ptab = table[parents.clamp(min=0)]
    kept = at < full[:, None]
    refs = refs - torch.bincount(table[at < -(-lens // page)[:, None]], minlength=N)
    refs = refs + torch.bincount(ptab[kept], minlength=N)
    last = ptab.gather(1, full.clamp(max=M - 1)[:, None]).squeeze(1).clamp(min=0)
    first = torch.full((N,), B, device=DEV).scatter_reduce(0, last, torch.where(cut, child, B), "amin")
    owns = cut & (refs[last] == 0) & (first[last] == child)
    refs = refs.scatter_add(0, last, owns.long())
    have = full + owns.long()
    held = -(-s["new"].long() // page)
    need = held - have
    start = need.cumsum(0) - need
    order = (refs > 0).to(torch.uint8).argsort(stable=True)  # free pages first, lowest first
    total, free = need.sum(), (refs == 0).sum()
    refs = refs.scatter_add(0, order, (torch.arange(N, device=DEV) < total).long())
    new = order[(start[:, None] + at - have[:, None]).clamp(0, N - 1)]
    out = torch.where(at < have[:, None], ptab, torch.where(at < held[:, None], new, -1))
    i = (cut & ~owns).nonzero().squeeze(1)
    token = torch.arange(page, device=DEV)
    row, slot = (token < (keep[i] % page)[:, None]).nonzero(as_tuple=True)
    src, dst = last[i][row], out[i, full[i]][row]
    for x in _caches(s):
        x[:, dst, slot] = x[:, src, slot]
    info = torch.stack([free - total, torch.zeros_like(total)])
    return s["k"], s["v"], s["ks"], s["vs"], out.int(), s["new"].clone(), refs.int(), info.int()


def _plain_compact(s):
    N = s["case"]["pages"]
    ids = torch.arange(N, device=DEV)
    live = s["refs"] > 0
    n_live = live.sum()
    before = live.cumsum(0) - live.long()
    low = (live & (ids < n_live)).sum()
    slots = live.to(torch.uint8).argsort(stable=True)  # free slots first, lowest first
    moved = live & (ids >= n_live)
    page_map = torch.where(live, torch.where(moved, slots[(before - low).clamp(min=0)], ids), -1)
    table = torch.where(s["table"] >= 0, page_map[s["table"].long().clamp(min=0)], -1)
    refs = torch.zeros_like(s["refs"])
    refs[page_map[live]] = s["refs"][live]
    src = moved.nonzero().squeeze(1)
    for x in _caches(s):
        x[:, page_map[src]] = x[:, src]
    return s["k"], s["v"], s["ks"], s["vs"], table.int(), refs, page_map.int(), torch.stack([n_live, moved.sum()]).int()


# ------------------------------------------------------------------------------------ the calls

def _own_run(s):
    from exact_long_context_tmem_b200 import attn as A

    op = s["op"]
    sc = dict(k_scale=s["ks"], v_scale=s["vs"])
    if op == "tree":
        if s["table"] is None:
            return A.attn_decode_tree(s["q"], s["k"], s["v"], s["lens"], s["mask"], q_lens=s["q_lens"], **sc)
        return A.attn_decode_tree_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], s["mask"], q_lens=s["q_lens"],
                                        **sc)
    if op == "accept":
        lens = A.attn_tree_accept(s["k"], s["v"], s["lens"], s["path"], s["n_acc"], n_q=s["case"]["n_q"],
                                  page_table=s["table"], **sc)
        return s["k"], s["v"], s["ks"], s["vs"], lens
    if op == "copy":
        A.attn_pages_copy(s["k"], s["v"], s["src"], s["dst"], **sc)
        return s["k"], s["v"], s["ks"], s["vs"]
    if op == "fork":
        return (s["k"], s["v"], s["ks"], s["vs"]) + tuple(A.attn_pages_fork(
            s["k"], s["v"], s["table"], s["lens"], s["refs"], s["parents"], keep_lens=s["keep"], new_lens=s["new"],
            **sc))
    return (s["k"], s["v"], s["ks"], s["vs"]) + tuple(A.attn_pages_compact(s["k"], s["v"], s["table"], s["refs"],
                                                                           **sc))


PLAIN = {"tree": _plain_tree, "accept": _plain_accept, "copy": _plain_copy, "fork": _plain_fork,
         "compact": _plain_compact}


def run(state):
    return _own_run(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------------ what it takes

def work(case):
    op, Hkv, D = case["op"], case["Hkv"], case["D"]
    token = 2 * Hkv * (D * ROW[case["kv"]] + (4 if case["kv"] != "bf16" else 0))  # K and V rows, with their scales
    if op == "tree":
        lens, q_lens = _tree_lens(case)
        rows = case["B"] * case["n_q"] * case["Hq"]
        seen = sum(q * (n - q) + q * (q + 1) / 2 for n, q in zip(lens, q_lens))
        table = 4 * sum(-(-n // case["page"]) for n in lens) if case["paged"] else 0
        return dict(bytes=sum(lens) * token + rows * (4 * D + 4) + case["B"] * (8 * case["n_q"] + 8) + table,
                    flops=4.0 * D * case["Hq"] * seen)
    if op == "accept":
        acc, _ = _accept_lists(case, _shape_rng(case))
        moved = sum(sum(i != j for j, i in enumerate(a)) for a in acc)
        return dict(bytes=2 * moved * token * case["L"] + case["B"] * (12 + 4 * case["n_q"]), flops=0)
    token *= case["L"]
    if op == "copy":
        return dict(bytes=2 * case["n"] * case["page"] * token + 8 * case["n"], flops=0)
    page, N = case["page"], case["pages"]
    if op == "fork":
        lens, table, refs, parents, keep, new, width = _fork_lists(case)
        copied, first, after = 0, set(), list(refs)
        for row, n in zip(table, lens):
            for p in row[:-(-n // page)]:
                after[p] -= 1
        for p, k in zip(parents, keep):
            for x in (table[p][:k // page] if p >= 0 else []):
                after[x] += 1
        for p, k in zip(parents, keep):
            if p >= 0 and k % page:
                x = table[p][k // page]
                if after[x] or x in first:
                    copied += k % page
                first.add(x)
        return dict(bytes=2 * copied * token + 8 * case["B"] * width + 8 * N + 24 * case["B"], flops=0)
    _, lens, table, refs, width = _pool_lists(case)
    n_live = sum(x > 0 for x in refs)
    moved = sum(x > 0 for x in refs[n_live:])
    return dict(bytes=2 * moved * page * token + 8 * case["B"] * width + 12 * N, flops=0)


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """Attention of the drafted tokens by its definition, sequence by sequence; what the other operators return is
    moved and counted, not computed."""
    if case["op"] != "tree":
        return None
    s = prepare(case, seed)
    B, n, Hq, Hkv, D, page = case["B"], case["n_q"], case["Hq"], case["Hkv"], case["D"], case["page"]
    G = Hq // Hkv
    o = torch.zeros(B, n, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, n, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, (length, q_len) in enumerate(zip(s["lens"].tolist(), s["q_lens"].tolist())):
        slots = torch.arange(length, device=DEV)
        if s["table"] is not None:
            where = (s["table"][b].long()[slots // page], slots % page)
        else:
            where = (torch.full_like(slots, b), slots)
        base = length - q_len
        sees = torch.ones(q_len, length, dtype=torch.bool, device=DEV)
        for i, m in enumerate(s["mask"][b, :q_len].tolist()):
            sees[i, base:] = torch.tensor([bool(m >> j & 1) for j in range(q_len)], device=DEV)
        for h in range(Hkv):
            keys, vals = (_exact_values(s[c][where[0], where[1], h],
                                        None if s[c + "s"] is None else s[c + "s"][where[0], where[1], h], case["kv"])
                          for c in "kv")
            heads = slice(h * G, (h + 1) * G)
            x = torch.einsum("igd,td->igt", s["q"][b, :q_len, heads].double(), keys) / math.sqrt(D)
            x = torch.where(sees[:, None], x, -math.inf)
            lse[b, :q_len, heads] = x.logsumexp(-1)
            o[b, :q_len, heads] = torch.einsum("igt,td->igd", x.softmax(-1), vals)
    return o, lse


def _exact_values(codes, scale, kv):
    if kv == "bf16":
        return codes.double()
    if kv == "fp8":
        c = codes.long()
        e, m = (c >> 3) & 15, (c & 7).double()
        x = torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7).double(), m * 2.0 ** -9)
        x = torch.where(c >= 128, -x, x)
    elif kv == "int8":
        x = codes.double()
    else:
        lo, hi = codes.long() % 16, codes.long() // 16
        x = torch.stack([lo, hi], -1).flatten(-2).double()
        x = torch.where(x >= 8, x - 16, x)
    return x * scale.double()[..., None]
