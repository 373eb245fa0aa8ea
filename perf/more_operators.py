"""The operators of a step that verifies drafted tokens over the paged cache, timed case by case.

A drafting model proposes a tree of tokens per sequence; the target model scores every node in one step, and the path
that it agrees with stays in the cache.  Four operators, on the two attention layer types of the package (sliding: 16
query heads over 8 KV heads of 256 dims, window 1024; global: 16 query heads over 1 KV head of 512 dims), bf16 pages of
16 positions:

  pages   the block tables of a step, from the requests' lengths: pages taken from a free list and given back to it
  append  head norms, position rotation and cache write of the nodes: each at its own slot, turned at its depth
  tree    attention of the nodes over the cached context and their own ancestors
  commit  the keys and values of the accepted path moved to consecutive positions, in all layers of a type

A tree is an int32 per node: the node of the same sequence that it continues, -1 for one that continues the context.
``run`` computes the plain form (elementary torch operations in 32 bits) or, with ``own`` set, makes the package's calls.
``exact`` is the definition in 64 bits.  Every pass leaves the state as the next one finds it.
"""

import math
import random

import torch

own = False

DEV = "cuda"
PAGE = 16
EPS = 1e-6
HEADS = {"sliding": (16, 8, 256), "global": (16, 1, 512)}  # query heads, KV heads, head dim
ROPE = {"sliding": (1.0e4, 128), "global": (1.0e6, 64)}    # theta, rotated pairs (i, i + D/2)
WINDOW = {"sliding": 1024, "global": 0}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one user, a short text, a short tree: what a call costs at least
        dict(name="tree-global-1x4", op="tree", kind="global", batch=1, n_lo=4, n_hi=4, ctx_lo=900, ctx_hi=900,
             lens_seed=21),
        # a few users with trees of odd sizes behind texts of any length
        dict(name="tree-global-8-ragged", op="tree", kind="global", batch=8, n_lo=3, n_hi=19, ctx_lo=0, ctx_hi=8192,
             lens_seed=22),
        # long contexts, small trees: bound by reading the cache
        dict(name="tree-global-16x131072", op="tree", kind="global", batch=16, n_lo=8, n_hi=8, ctx_lo=131072,
             ctx_hi=131072, lens_seed=23),
        # wide trees: bound by the products
        dict(name="tree-global-32-wide", op="tree", kind="global", batch=32, n_lo=64, n_hi=64, ctx_lo=4000,
             ctx_hi=8192, lens_seed=24),
        # the smallest sliding call
        dict(name="tree-sliding-4-short", op="tree", kind="sliding", batch=4, n_lo=1, n_hi=9, ctx_lo=0, ctx_hi=1100,
             lens_seed=25),
        # a full verification batch on a sliding layer, trees of 17 to 45 nodes
        dict(name="tree-sliding-64-ragged", op="tree", kind="sliding", batch=64, n_lo=17, n_hi=45, ctx_lo=1024,
             ctx_hi=32768, lens_seed=26),
        # the nodes of one user on a global layer: latency
        dict(name="append-global-1x7", op="append", kind="global", batch=1, n_lo=7, n_hi=7, ctx_lo=20000,
             ctx_hi=20000, lens_seed=27),
        # the nodes of a full batch on a sliding layer
        dict(name="append-sliding-64-ragged", op="append", kind="sliding", batch=64, n_lo=17, n_hi=45, ctx_lo=1024,
             ctx_hi=32768, lens_seed=28),
        # one user's accepted path in the global layers
        dict(name="commit-global-1", op="commit", kind="global", batch=1, n_lo=13, n_hi=13, ctx_lo=4000, ctx_hi=4000,
             layers=8, lens_seed=35),
        # a full batch's accepted paths in the sliding layers
        dict(name="commit-sliding-64", op="commit", kind="sliding", batch=64, n_lo=17, n_hi=45, ctx_lo=1024,
             ctx_hi=32768, layers=40, lens_seed=30),
        # one step of a running batch: a page here and there
        dict(name="pages-step-64", op="pages", kind="sliding", batch=64, n_lo=17, n_hi=45, ctx_lo=1024, ctx_hi=32768,
             finished=0.0, admitted=0.0, prompt_hi=1, lens_seed=31),
        # prompts admitted and finished requests' pages given back, next to running ones
        dict(name="pages-prompts-200", op="pages", kind="global", batch=200, n_lo=1, n_hi=64, ctx_lo=0, ctx_hi=65536,
             finished=0.2, admitted=0.3, prompt_hi=32768, lens_seed=32),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "append", "commit", "pages"])
    kind = rng.choice(["sliding", "global"])
    c = dict(op=op, kind=kind, lens_seed=rng.randrange(1 << 20))
    if op == "tree":
        c["n_hi"] = _log(rng, 1, 64)
        c["batch"] = _log(rng, 1, 64)
        most = 32768 if kind == "sliding" else min(131072, (1 << 20) // c["batch"],
                                                   (1 << 23) // (c["batch"] * c["n_hi"]))
        c["ctx_hi"] = _log(rng, 1, most)
    elif op == "append":
        c["n_hi"] = _log(rng, 1, 64)
        c["batch"] = _log(rng, 1, 100)
        c["ctx_hi"] = _log(rng, 1, 200000)
    elif op == "commit":
        c["n_hi"] = rng.randint(2, 64)
        c["batch"] = _log(rng, 1, 64)
        c["ctx_hi"] = _log(rng, 1, 32768)
        c["layers"] = rng.randint(1, 40 if kind == "sliding" else 8)
    else:
        c["n_hi"] = _log(rng, 1, 64)
        c["batch"] = _log(rng, 1, 256)
        c["ctx_hi"] = _log(rng, 1, 32768)
        c["finished"] = rng.choice([0.0, round(rng.uniform(0.0, 0.3), 3)])
        c["admitted"] = rng.choice([0.0, round(rng.uniform(0.0, 0.3), 3)])
        c["prompt_hi"] = _log(rng, 1, 32768)
    c["n_lo"] = rng.randint(1 if op != "commit" else 2, c["n_hi"])
    c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
    return c


def _lengths(case):
    """(context lengths, nodes) of the sequences; the first has the most of both."""
    r = random.Random(case["lens_seed"])
    B = case["batch"]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(B)]
    n = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(B)]
    ctx[0], n[0] = case["ctx_hi"], case["n_hi"]
    return ctx, n


def _keep(kind, cached):
    """First position that a node behind `cached` tokens sees."""
    w = WINDOW[kind]
    return max(0, cached - w + 1) if w > 0 else 0


def _requests(case):
    """Per request of a pages case: (cached, new tokens, logical pages held before: first, end)."""
    r = random.Random(case["lens_seed"] + 1)
    out = []
    for c, n in zip(*_lengths(case)):
        u = r.random()
        if u < case["admitted"]:
            out.append((0, r.randint(1, case["prompt_hi"]), 0, 0))
            continue
        # the step before held pages for its own nodes behind fewer accepted tokens
        before = max(0, c - r.randint(1, 6))
        first = _keep(case["kind"], before) // PAGE
        end = max(first, -(-(before + r.randint(case["n_lo"], case["n_hi"])) // PAGE))
        if u < case["admitted"] + case["finished"]:
            out.append((0, 0, first, end))
        else:
            out.append((c, n, first, end))
    return out


def _page_range(kind, cached, new):
    first = _keep(kind, cached) // PAGE
    return first, max(first, -(-(cached + new) // PAGE))


def _table_width(case):
    return max(1, max(max(e, _page_range(case["kind"], c, n)[1]) for c, n, _, e in _requests(case)))


def work(case):
    Hq, Hkv, D = HEADS[case["kind"]]
    op = case["op"]
    if op == "pages":
        moved = 0
        for c, n, f, e in _requests(case):
            g, h = _page_range(case["kind"], c, n)
            both = max(0, min(e, h) - max(f, g))
            moved += (e - f) + (h - g) - 2 * both
        # a page given back or taken: an entry of the table and one of the free list
        return {"bytes": 8 * moved + 4 * (8 * case["batch"] + 5), "flops": 8 * case["batch"] + moved}
    ctx, n = _lengths(case)
    T = sum(n)
    if op == "append":
        row = Hq * D + (D if case["kind"] == "global" else 2 * Hkv * D)
        return {"bytes": T * (2 * row + 2 * Hq * D + 2 * Hkv * D * 2 + 4) + 4 * D,
                "flops": T * ((Hq + 2 * Hkv) * D * 4 + (Hq + Hkv) * ROPE[case["kind"]][1] * 6)}
    if op == "commit":
        moved = sum(sum(1 for j, s in enumerate(p) if s != j) for p in _paths(case))
        return {"bytes": moved * case["layers"] * 2 * 2 * Hkv * D * 2 + 4 * T, "flops": moved}
    w = WINDOW[case["kind"]]
    seen = sum(c + m - _keep(case["kind"], c) for c, m in zip(ctx, n))
    # a node sees the context's window and at least itself (ancestors aside)
    pairs = sum(m * ((min(c, w - 1) if w > 0 else c) + 1) for c, m in zip(ctx, n))
    return {"bytes": seen * 2 * Hkv * D * 2 + 2 * T * Hq * D * 2 + 4 * T, "flops": pairs * Hq * D * 4}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _unit(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _weight(D, gen):
    # norm weights that give logits of a standard deviation near 2.5, as trained ones do (no further scale)
    return ((1.0 + 0.1 * torch.randn(D, generator=gen, device=DEV)) * math.sqrt(2.5) / D ** 0.25).to(torch.bfloat16)


def _rows(rows, D, gen, w=None):
    """Cache rows [rows, D] of a filled cache, in pieces."""
    out = torch.empty((rows, D), dtype=torch.bfloat16, device=DEV)
    step = 1 << 18
    for r in range(0, rows, step):
        x = _unit(torch.randn((min(step, rows - r), D), generator=gen, device=DEV))
        out[r:r + step] = x if w is None else x * w.float()
    return out


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _parents(n, rng):
    """A tree of n nodes in the order they were drafted: a node continues an earlier one, most often a late one."""
    out = []
    for i in range(n):
        if i == 0:
            out.append(-1)
        else:
            out.append(max(i - 1 - int(rng.expovariate(0.35)), 0 if rng.random() < 0.98 else -1))
    return out


def _paths(case):
    """Accepted nodes of each sequence: a few first ones in place, the others from behind the path's end."""
    r = random.Random(case["lens_seed"] + 2)
    out = []
    for n in _lengths(case)[1]:
        k = r.randint(1, max(1, min(8, n // 2)))
        still = r.randint(0, k)
        out.append(list(range(still)) + sorted(r.sample(range(k, n), min(k - still, n - k))))
    return out


def _pages_state(case, seed, host):
    B, P = case["batch"], 0
    req = _requests(case)
    width = _table_width(case)
    held = sum(e - f for _, _, f, e in req)
    need = sum(max(0, _page_range(case["kind"], c, n)[1] - _page_range(case["kind"], c, n)[0]) for c, n, _, _ in req)
    P = held + need + 100
    perm = torch.randperm(P, generator=host).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, (_, _, f, e) in enumerate(req):
        table[b, f:e] = perm[at:at + e - f]
        at += e - f
    head = int(torch.randint(0, P, (1,), generator=host))
    ring = torch.full((P,), -1, dtype=torch.int32)
    ring[(head + torch.arange(P - at)) % P] = perm[at:]
    s = dict(op="pages", kind=case["kind"], num_pages=P, window=WINDOW[case["kind"]])
    s["cached"], s["new"] = _int32([x[0] for x in req]), _int32([x[1] for x in req])
    s["held"] = _int32([[x[2], x[3]] for x in req])
    s["free_state"] = _int32([head, P - at])
    s["table"], s["free_list"] = table.to(DEV), ring.to(DEV)
    s["seq_lens"], s["cu_q"] = _int32([0] * B), _int32([0] * (B + 1))
    s["held_out"], s["free_state_out"] = torch.zeros_like(s["held"]), torch.zeros_like(s["free_state"])
    return s


def prepare(case, seed):
    kind, op = case["kind"], case["op"]
    Hq, Hkv, D = HEADS[kind]
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    rng = random.Random(int(seed))
    if op == "pages":
        return _pages_state(case, seed, host)
    ctx, n = _lengths(case)
    L = [c + m for c, m in zip(ctx, n)]
    T = sum(n)
    s = dict(op=op, kind=kind, max_len=max(L), max_n=max(n), layers=case.get("layers", 1))
    s["seq_lens"] = _int32(L)
    cu = [0]
    for m in n:
        cu.append(cu[-1] + m)
    s["cu_q"] = _int32(cu)
    # pages of the positions that the call touches
    first = [_keep(kind, c) if op == "tree" else c for c in ctx]
    need = [(f // PAGE, -(-x // PAGE)) for f, x in zip(first, L)]
    P = sum(e - f for f, e in need)
    perm = torch.randperm(P, generator=host).to(torch.int32)
    table = torch.full((len(L), -(-max(L) // PAGE)), -1, dtype=torch.int32)
    at = 0
    for b, (f, e) in enumerate(need):
        table[b, f:e] = perm[at:at + e - f]
        at += e - f
    s["table"] = table.to(DEV)
    if op in ("tree", "append"):
        s["parents"] = _int32([p for m in n for p in _parents(m, rng)])
    w_k = _weight(D, gen)
    layers = s["layers"]
    for name, w in (("k_pool", w_k), ("v_pool", None)):
        s[name] = _rows(layers * P * PAGE * Hkv, D, gen, w).view(layers, P, PAGE, Hkv, D)
    if op == "append":
        s["qkv"] = torch.randn((T, Hq * D + (D if kind == "global" else 2 * Hkv * D)), generator=gen,
                               device=DEV).to(torch.bfloat16)
        s["w_q"], s["w_k"] = _weight(D, gen), _weight(D, gen)
        s["q_out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    elif op == "tree":
        s["q"] = (_unit(torch.randn((T, Hq, D), generator=gen, device=DEV)) * _weight(D, gen).float()).to(torch.bfloat16)
        s["o"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    else:
        paths = _paths(case)
        width = max(len(p) for p in paths)
        s["path"] = _int32([p + [0] * (width - len(p)) for p in paths])
        s["path_len"] = _int32([len(p) for p in paths])
        s["new_lens"] = _int32([0] * len(L))
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_tree(s):
    """(packed row of node [B, N], which exist, depth [B, N], ancestors or self [B, N, N]) from the parents."""
    cu = s["cu_q"].long()
    n = cu[1:] - cu[:-1]
    node = torch.arange(s["max_n"], device=DEV)
    there = node < n[:, None]
    row = (cu[:-1, None] + node).clamp(max=s["parents"].shape[0] - 1)
    parent = torch.where(there, s["parents"].long()[row], torch.full_like(row, -1))
    reach = ((parent[:, :, None] == node) | (node[:, None] == node)).float()
    for _ in range(max(1, (s["max_n"] - 1).bit_length())):
        reach = (torch.matmul(reach, reach) > 0).float()
    reach = (reach > 0) & there[:, :, None]
    return row, there, reach.sum(-1) - 1, reach


def _plain_attention(s):
    Hq, Hkv, D = HEADS[s["kind"]]
    w = WINDOW[s["kind"]]
    row, there, depth, reach = _plain_tree(s)
    B, N = row.shape
    L = s["seq_lens"].long()
    ctx = L - there.sum(-1)
    W = min(s["max_len"], w + N) if w > 0 else s["max_len"]
    slot = L[:, None] - W + torch.arange(W, device=DEV)         # cache positions of each sequence's last W
    first = (ctx - w + 1).clamp(min=0) if w > 0 else torch.zeros_like(ctx)
    held = slot >= first[:, None]
    pos = slot.clamp(min=0)
    seq = torch.arange(B, device=DEV)[:, None]
    at = (s["table"][seq, pos // PAGE].long() * PAGE + pos % PAGE).clamp(min=0)
    at = torch.where(held, at, torch.zeros_like(at))
    as_node = (slot - ctx[:, None])                             # < 0: context
    seen = torch.gather(reach, 2, as_node.clamp(min=0)[:, None].expand(B, N, W))
    where = torch.where(as_node < 0, slot, ctx[:, None] + torch.gather(depth, 1, as_node.clamp(min=0)))
    seen = held[:, None] & ((as_node < 0)[:, None] | seen) & there[:, :, None]
    if w > 0:
        seen &= where[:, None] > (ctx[:, None] + depth - w)[:, :, None]
    q = s["q"].float()[row].view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    k = s["k_pool"].view(-1, Hkv, D)[at].float().permute(0, 2, 3, 1)
    x = torch.matmul(q, k).view(B, Hkv, Hq // Hkv, N, W).masked_fill_(~seen[:, None, None], -math.inf)
    del k
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    v = s["v_pool"].view(-1, Hkv, D)[at].float().transpose(1, 2)
    o = torch.matmul(x.view(B, Hkv, -1, W), v) / x.sum(-1).view(B, Hkv, -1, 1).clamp(min=1e-30)
    o = o.view(B, Hkv, Hq // Hkv, N, D).permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)
    # the nodes' rows in their packed order
    T = s["q"].shape[0]
    token = torch.arange(T, device=DEV)
    b = torch.searchsorted(s["cu_q"][1:].long(), token, right=True)
    s["o"].copy_(o[b, token - s["cu_q"].long()[b]])
    return s["o"]


def _plain_append(s):
    Hq, Hkv, D = HEADS[s["kind"]]
    theta, pairs = ROPE[s["kind"]]
    T = s["qkv"].shape[0]
    _, there, depths, _ = _plain_tree(s)
    token = torch.arange(T, device=DEV)
    seq = torch.searchsorted(s["cu_q"][1:].long(), token, right=True)
    node = token - s["cu_q"].long()[seq]
    ctx = (s["seq_lens"].long() - there.sum(-1))[seq]
    x = s["qkv"].float()
    q = _unit(x[:, :Hq * D].view(T, Hq, D)) * s["w_q"].float()
    kv = x[:, Hq * D:].view(T, -1, Hkv, D)
    k = _unit(kv[:, 0]) * s["w_k"].float()
    v = _unit(kv[:, -1])
    freq = theta ** (-2.0 * torch.arange(pairs, device=DEV, dtype=torch.float64) / D)
    angle = (ctx + depths[seq, node]).double()[:, None, None] * freq  # far positions: in 64 bits
    c, sn = torch.cos(angle).float(), torch.sin(angle).float()
    half = D // 2
    out = []
    for y in (q, k):
        a, b = y[..., :pairs], y[..., half:half + pairs]
        out.append(torch.cat([a * c - b * sn, y[..., pairs:half], b * c + a * sn, y[..., half + pairs:]], -1))
    q, k = out
    s["q_out"].copy_(q)
    pos = ctx + node
    slot = s["table"][seq, pos // PAGE].long() * PAGE + pos % PAGE
    s["k_pool"].view(-1, Hkv, D)[slot] = k.to(torch.bfloat16)
    s["v_pool"].view(-1, Hkv, D)[slot] = v.to(torch.bfloat16)
    return s["q_out"], s["k_pool"], s["v_pool"]


def _plain_commit(s):
    cu = s["cu_q"].long()
    ctx = s["seq_lens"].long() - (cu[1:] - cu[:-1])
    B, width = s["path"].shape
    j = torch.arange(width, device=DEV)
    taken = j < s["path_len"][:, None]
    src = ctx[:, None] + torch.where(taken, s["path"].long(), torch.zeros_like(s["path"].long()))
    dst = torch.where(taken, ctx[:, None] + j, src)             # rows behind a path stay what they are
    seq = torch.arange(B, device=DEV)[:, None]
    src, dst = (s["table"][seq, p // PAGE].long() * PAGE + p % PAGE for p in (src, dst))
    src, dst = src[taken], dst[taken]
    for pool in (s["k_pool"], s["v_pool"]):
        x = pool.view(pool.shape[0], -1, pool.shape[3] * pool.shape[4])
        x[:, dst] = x[:, src]
    s["new_lens"].copy_(ctx + s["path_len"])
    return s["k_pool"], s["v_pool"], s["new_lens"]


def _plain_pages(s):
    cached, new, held = s["cached"].long(), s["new"].long(), s["held"].long()
    head, count = s["free_state"].long()
    P = s["num_pages"]
    w = s["window"]
    first = (cached - w + 1).clamp(min=0) // PAGE if w > 0 else torch.zeros_like(cached)
    end = torch.maximum(first, (cached + new + PAGE - 1) // PAGE)
    lp = torch.arange(s["table"].shape[1], device=DEV)
    had = (lp >= held[:, :1]) & (lp < held[:, 1:])
    has = (lp >= first[:, None]) & (lp < end[:, None])
    give, take = (had & ~has).flatten(), (has & ~had).flatten()
    given, taken = torch.cumsum(give, 0), torch.cumsum(take, 0)
    table = s["table"].flatten().long()
    fetched = s["free_list"].long()[(head + taken - 1) % P]
    # what is given back goes behind the free pages; every other entry into a row that is dropped
    ring = torch.cat([s["free_list"], s["free_list"][:1]])
    ring[torch.where(give, (head + count + given - 1) % P, torch.full_like(given, P))] = table.to(torch.int32)
    s["free_list"].copy_(ring[:P])
    s["table"].copy_(torch.where(take, fetched, table).view(s["table"].shape))
    s["held_out"].copy_(torch.stack([first, end], 1))
    s["free_state_out"].copy_(torch.stack([(head + taken[-1]) % P, count - taken[-1] + given[-1]]))
    s["seq_lens"].copy_(cached + new)
    s["cu_q"][1:] = torch.cumsum(new, 0)
    return s["table"], s["held_out"], s["free_list"], s["free_state_out"], s["seq_lens"], s["cu_q"]


# ---------------------------------------------------------------------------
# the package's calls: prepared once per state, as a serving loop keeps them
# ---------------------------------------------------------------------------

def _prepared(s):
    import paged_decode_attention_gb300 as pda

    if s["op"] == "pages":
        call = pda.prepare_pages_assign(s["cached"], s["new"], s["table"], s["held"], s["free_list"], s["free_state"],
                                        s["seq_lens"], s["cu_q"], window=s["window"], held_out=s["held_out"],
                                        free_state_out=s["free_state_out"])
        return call, (s["table"], s["held_out"], s["free_list"], s["free_state_out"], s["seq_lens"], s["cu_q"])
    kind = s["kind"]
    if s["op"] == "tree":
        fn = getattr(pda, "prepare_decode_%s_tree" % kind)
        return fn(s["q"], s["k_pool"][0], s["v_pool"][0], s["table"], s["seq_lens"], s["cu_q"], s["parents"], s["o"],
                  max_q=s["max_n"], max_seq_len=s["max_len"]), s["o"]
    if s["op"] == "append":
        fn = getattr(pda, "prepare_kv_append_%s_tree" % kind)
        return fn(s["qkv"], s["w_q"], s["w_k"], s["table"], s["seq_lens"], s["cu_q"], s["parents"], s["k_pool"][0],
                  s["v_pool"][0], s["q_out"]), (s["q_out"], s["k_pool"], s["v_pool"])
    fn = getattr(pda, "prepare_kv_commit_%s" % kind)
    return fn(list(s["k_pool"]), list(s["v_pool"]), s["table"], s["seq_lens"], s["cu_q"], s["path"], s["path_len"],
              s["new_lens"]), (s["k_pool"], s["v_pool"], s["new_lens"])


def run(state):
    if own:
        if "call" not in state:
            state["call"], state["out"] = _prepared(state)
        state["call"].run(torch.cuda.current_stream())
        return state["out"]
    return {"tree": _plain_attention, "append": _plain_append, "commit": _plain_commit,
            "pages": _plain_pages}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _chains(s, case):
    """Per sequence: the list of every node's ancestors, itself included, by walking up."""
    parents = s["parents"].tolist()
    out, at = [], 0
    for m in _lengths(case)[1]:
        chains = []
        for i in range(m):
            p = parents[at + i]
            chains.append(([] if p < 0 else chains[p]) + [i])
        out.append(chains)
        at += m
    return out


def _slot(s, b, positions):
    return s["table"][b][positions // PAGE].long(), positions % PAGE


def _exact_tree(s, case):
    Hq, Hkv, D = HEADS[s["kind"]]
    G, w = Hq // Hkv, WINDOW[s["kind"]]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (c, m, chains) in enumerate(zip(*_lengths(case), _chains(s, case))):
        lo = _keep(s["kind"], c)
        seen = torch.zeros((m, c + m - lo), dtype=torch.bool)
        for i, chain in enumerate(chains):
            here = c + len(chain) - 1
            seen[i, max(0, (here - w + 1 if w > 0 else 0) - lo):c - lo] = True
            for a in chain:
                if w <= 0 or len(chain) - len(chains[a]) < w:
                    seen[i, c - lo + a] = True
        seen = seen.to(DEV).repeat_interleave(G, 0)
        page, row = _slot(s, b, torch.arange(lo, c + m, device=DEV))
        for h in range(Hkv):
            k, v = (s[x][0][page, row, h].double() for x in ("k_pool", "v_pool"))
            q = s["q"][at:at + m, h * G:(h + 1) * G].double().reshape(m * G, D)
            p = torch.softmax((q @ k.t()).masked_fill(~seen, -math.inf), -1)
            o[at:at + m, h * G:(h + 1) * G] = (p @ v).view(m, G, D)
        at += m
    return o


def _exact_append(s, case):
    Hq, Hkv, D = HEADS[s["kind"]]
    theta, pairs = ROPE[s["kind"]]
    ctx, n = _lengths(case)
    turn_at, page, row = [], [], []
    for b, (c, m, chains) in enumerate(zip(ctx, n, _chains(s, case))):
        turn_at += [c + len(chain) - 1 for chain in chains]
        p, r = _slot(s, b, torch.arange(c, c + m, device=DEV))
        page.append(p)
        row.append(r)
    page, row = torch.cat(page), torch.cat(row)
    pos = torch.tensor(turn_at, dtype=torch.float64, device=DEV)
    x = s["qkv"].double()
    T = x.shape[0]
    i = torch.arange(D // 2, device=DEV).double()
    turn = torch.where(i < pairs, torch.exp(-2.0 * i / D * math.log(theta)), torch.zeros_like(i))
    spin = torch.polar(torch.ones_like(turn)[None, None], pos[:, None, None] * turn)

    def norm(y):
        return y / ((y * y).sum(-1, keepdim=True) / y.shape[-1] + EPS).sqrt()

    def rotated(y):
        z = torch.complex(y[..., :D // 2].contiguous(), y[..., D // 2:].contiguous()) * spin
        return torch.cat([z.real, z.imag], -1)

    q = rotated(norm(x[:, :Hq * D].reshape(T, Hq, D)) * s["w_q"].double())
    k, v = s["k_pool"].double(), s["v_pool"].double()
    k[0][page, row] = rotated(norm(x[:, Hq * D:Hq * D + Hkv * D].reshape(T, Hkv, D)) * s["w_k"].double())
    v[0][page, row] = norm(x[:, -Hkv * D:].reshape(T, Hkv, D))
    return q, k, v


def _exact_commit(s, case):
    ctx, _ = _lengths(case)
    pools = [s["k_pool"].clone(), s["v_pool"].clone()]
    paths = _paths(case)
    for b, path in enumerate(paths):
        src = [x.tolist() for x in _slot(s, b, torch.tensor([ctx[b] + p for p in path], device=DEV))]
        dst = [x.tolist() for x in _slot(s, b, torch.arange(ctx[b], ctx[b] + len(path), device=DEV))]
        for j in range(len(path)):
            for x, old in zip(pools, (s["k_pool"], s["v_pool"])):
                x[:, dst[0][j], dst[1][j]] = old[:, src[0][j], src[1][j]]
    return pools[0], pools[1], _int32([c + len(p) for c, p in zip(ctx, paths)])


def _exact_pages(s, case):
    table, free = s["table"].tolist(), s["free_list"].tolist()
    head, count = s["free_state"].tolist()
    P = len(free)
    req = _requests(case)
    held, lens, cu = [], [], [0]
    taken = given = 0
    for b, (c, n, f, e) in enumerate(req):
        g, h = _page_range(case["kind"], c, n)
        for lp in range(f, e):
            if not g <= lp < h:
                free[(head + count + given) % P] = table[b][lp]
                given += 1
        held.append([g, h])
        lens.append(c + n)
        cu.append(cu[-1] + n)
    for b, (c, n, f, e) in enumerate(req):
        for lp in range(*held[b]):
            if not f <= lp < e:
                table[b][lp] = free[(head + taken) % P]
                taken += 1
    return (_int32(table), _int32(held), _int32(free), _int32([(head + taken) % P, count - taken + given]),
            _int32(lens), _int32(cu))


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "append": _exact_append, "commit": _exact_commit,
            "pages": _exact_pages}[case["op"]](s, case)
