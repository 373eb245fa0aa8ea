"""The operators of a serving step around the paged cache, timed case by case.

Five operators, on the two attention layer types of the package (sliding: 16 query heads over 8 KV heads of 256 dims,
window 1024; global: 16 query heads over 1 KV head of 512 dims), pages of 16 positions:

  append_chunk   head norms, position rotation and cache write of a ragged chunk of new tokens per sequence (bf16 cache)
  append_fp8     the same into an 8-bit cache: e4m3 values, one power-of-two scale per position and head
  read_fp8       an 8-bit cache read back into bf16 pages (what the multi-query attention takes)
  decode_fp8     one query per sequence over an 8-bit cache
  decode_prefix  one query per sequence over a prefix that the whole batch shares and a suffix of its own

``run`` computes the plain form (elementary torch operations in 32 bits) or, with ``own`` set, makes the package's calls.
``exact`` is the definition in 64 bits.
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
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a prompt batch: four prompts of 2048 tokens enter the sliding cache at once
        dict(name="append-chunk-sliding-4x2048", op="append_chunk", kind="sliding", batch=4, new_lo=2048, new_hi=2048,
             past_hi=0, lens_seed=1),
        # a mixed step of a scheduler: decode tokens and prompt pieces of odd lengths side by side
        dict(name="append-chunk-global-ragged", op="append_chunk", kind="global", batch=7, new_lo=1, new_hi=777,
             past_hi=20000, lens_seed=2),
        # one token for each of 64 sequences: the append of a decode step, where latency counts
        dict(name="append-fp8-sliding-step-64", op="append_fp8", kind="sliding", batch=64, new_lo=1, new_hi=1,
             past_hi=32768, lens_seed=3),
        # a piece of a long prompt late in its context
        dict(name="append-fp8-global-4096", op="append_fp8", kind="global", batch=1, new_lo=4096, new_hi=4096,
             past_hi=28672, lens_seed=4),
        # what a chunk of 1024 queries sees of eight sliding contexts: window + 1023 positions each
        dict(name="read-fp8-sliding-8x2047", op="read_fp8", kind="sliding", batch=8, len_lo=1500, len_hi=9000,
             span=2047, lens_seed=5),
        # a whole global context read back before a prompt piece attends to it
        dict(name="read-fp8-global-32768", op="read_fp8", kind="global", batch=1, len_lo=32768, len_hi=32768, span=0,
             lens_seed=6),
        # the smallest decode: four short sequences
        dict(name="decode-fp8-sliding-tiny", op="decode_fp8", kind="sliding", batch=4, len_lo=1, len_hi=1100,
             lens_seed=7),
        # a full decode batch on a sliding layer, window-only pages
        dict(name="decode-fp8-sliding-256", op="decode_fp8", kind="sliding", batch=256, len_lo=1024, len_hi=32768,
             lens_seed=8),
        # eight ragged global contexts
        dict(name="decode-fp8-global-8", op="decode_fp8", kind="global", batch=8, len_lo=1, len_hi=8192, lens_seed=9),
        # long contexts: sixteen of 131072 positions
        dict(name="decode-fp8-global-16x131072", op="decode_fp8", kind="global", batch=16, len_lo=131072,
             len_hi=131072, lens_seed=10),
        # a few users behind one system prompt of an odd length
        dict(name="decode-prefix-8", op="decode_prefix", kind="global", batch=8, prefix=5003, len_lo=1, len_hi=300,
             lens_seed=11),
        # many users behind one long document
        dict(name="decode-prefix-64", op="decode_prefix", kind="global", batch=64, prefix=32768, len_lo=1,
             len_hi=2048, lens_seed=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append_chunk", "append_fp8", "read_fp8", "decode_fp8", "decode_prefix"])
    kind = rng.choice(["sliding", "global"])
    c = dict(op=op, kind=kind, lens_seed=rng.randrange(1 << 20))
    if op in ("append_chunk", "append_fp8"):
        total = _log(rng, 1, 4096)
        c["batch"] = _log(rng, 1, min(256, total))
        mean = max(1, total // c["batch"])
        c["new_lo"] = rng.randint(1, mean)
        c["new_hi"] = 2 * mean - c["new_lo"]
        c["past_hi"] = rng.choice([0, _log(rng, 1, 200000)])
    elif op == "read_fp8":
        c["batch"] = _log(rng, 1, 64)
        c["span"] = rng.choice([0, _log(rng, 1, 4096)])
        c["len_hi"] = _log(rng, 1, max(1, 65536 // c["batch"]) * (2 if c["span"] else 1))
        c["len_lo"] = rng.randint(0, c["len_hi"])
    elif op == "decode_fp8":
        c["batch"] = _log(rng, 1, 256)
        c["len_hi"] = _log(rng, 1, 32768) if kind == "sliding" else _log(rng, 1, min(262144, (1 << 20) // c["batch"]))
        c["len_lo"] = rng.randint(0, c["len_hi"])
    else:
        c["kind"] = "global"
        c["batch"] = _log(rng, 1, 64)
        c["prefix"] = _log(rng, 1, 32768)
        c["len_hi"] = _log(rng, 1, 2048)
        c["len_lo"] = rng.randint(0, c["len_hi"])
    return c


def _lengths(case):
    """(cached tokens of each sequence, new tokens among them; None for the operators without)."""
    r = random.Random(case["lens_seed"])
    B = case["batch"]
    if "new_lo" in case:
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
        return [n + (case["past_hi"] if B == 1 else r.randint(0, case["past_hi"])) for n in new], new
    L = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(B)]
    L[0] = case["len_hi"]
    return L, None


def _first(case, L, new):
    """First position of a sequence that the call touches."""
    if new is not None:
        return L - new
    w = case.get("span", 0) if case["op"] == "read_fp8" else WINDOW[case["kind"]]
    return max(0, L - w) if w > 0 else 0


def work(case):
    Hq, Hkv, D = HEADS[case["kind"]]
    Ls, new = _lengths(case)
    op = case["op"]
    if new is not None:
        T = sum(new)
        row = Hq * D + (D if case["kind"] == "global" else 2 * Hkv * D)
        cache = 2 * Hkv * D * 2 if op == "append_chunk" else 2 * Hkv * (D + 1)
        # squares, scale and weight of every element; six operations for a rotated one, its angle aside
        return {"bytes": T * (2 * row + 2 * Hq * D + cache) + 4 * D,
                "flops": T * ((Hq + 2 * Hkv) * D * 4 + (Hq + Hkv) * ROPE[case["kind"]][1] * 6)}
    seen = sum(L - _first(case, L, None) for L in Ls)
    row = 2 * Hkv * (D + 1)
    if op == "read_fp8":
        return {"bytes": seen * (row + 2 * Hkv * D * 2), "flops": seen * 2 * Hkv * D}
    qo = 2 * case["batch"] * Hq * D * 2
    if op == "decode_fp8":
        return {"bytes": seen * row + qo, "flops": seen * Hq * D * 4}
    return {"bytes": (seen + case["prefix"]) * 2 * D * 2 + qo,
            "flops": (seen + case["prefix"] * case["batch"]) * Hq * D * 4}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _unit(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _quantised(x):
    """e4m3 values and power-of-two scales [..., 1] of the rows of x: the largest of a row lands in (224, 448]."""
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(-126, 127)
    return torch.ldexp(x, -k).to(F8), k


def _weight(D, gen):
    # norm weights that give logits of a standard deviation near 2.5, as trained ones do (no further scale)
    return ((1.0 + 0.1 * torch.randn(D, generator=gen, device=DEV)) * math.sqrt(2.5) / D ** 0.25).to(torch.bfloat16)


def _rows(rows, D, gen, w=None, fp8=False):
    """Cache rows of a filled cache, in pieces: (values [rows, D], scale exponents [rows] or None)."""
    out = torch.empty((rows, D), dtype=F8 if fp8 else torch.bfloat16, device=DEV)
    ks = torch.empty((rows,), dtype=torch.int32, device=DEV) if fp8 else None
    step = 1 << 18
    for r in range(0, rows, step):
        x = _unit(torch.randn((min(step, rows - r), D), generator=gen, device=DEV))
        x = x if w is None else x * w.float()
        if fp8:
            v, k = _quantised(x)
            out[r:r + step].view(torch.uint8).copy_(v.view(torch.uint8))
            ks[r:r + step] = k[:, 0]
        else:
            out[r:r + step] = x
    return out, ks


def _table(needed, width, gen):
    """Shuffled pages for the logical page ranges `needed` of each sequence: (table int32, number of pages)."""
    total = sum(max(0, b - a) for a, b in needed)
    perm = torch.randperm(total, generator=gen).to(torch.int32)
    t = torch.full((len(needed), max(1, width)), -1, dtype=torch.int32)
    at = 0
    for s, (a, b) in enumerate(needed):
        n = max(0, b - a)
        t[s, a:a + n] = perm[at:at + n]
        at += n
    return t.to(DEV), max(1, total)


def prepare(case, seed):
    kind, op = case["kind"], case["op"]
    Hq, Hkv, D = HEADS[kind]
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    Ls, new = _lengths(case)
    s = dict(op=op, kind=kind, max_len=max(Ls), span=case.get("span", 0))
    s["seq_lens"] = torch.tensor(Ls, dtype=torch.int32, device=DEV)
    pages = []
    for b, L in enumerate(Ls):
        a = _first(case, L, None if new is None else new[b])
        pages.append((a // PAGE, -(-L // PAGE) if L > a else a // PAGE))
    s["table"], P = _table(pages, -(-max(Ls) // PAGE), host)
    if new is not None:
        T = sum(new)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["qkv"] = torch.randn((T, Hq * D + (D if kind == "global" else 2 * Hkv * D)), generator=gen,
                               device=DEV).to(torch.bfloat16)
        s["w_q"], s["w_k"] = _weight(D, gen), _weight(D, gen)
        s["q_out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    fp8 = op in ("append_fp8", "read_fp8", "decode_fp8")
    w_k = _weight(D, gen)
    for name, w in (("k", w_k), ("v", None)):
        x, k = _rows(P * PAGE * Hkv, D, gen, w, fp8)
        s[name + "_pool"] = x.view(P, PAGE, Hkv, D)
        if fp8:
            k = (k + 127).to(torch.uint8).view(P, PAGE, Hkv).transpose(1, 2).contiguous()
            s[name + "_scale"] = k.view(E8)
    if op == "read_fp8":
        s["k_out"] = torch.zeros((P, PAGE, Hkv, D), dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.zeros((P, PAGE, Hkv, D), dtype=torch.bfloat16, device=DEV)
    if op in ("decode_fp8", "decode_prefix"):
        q = _unit(torch.randn((len(Ls), Hq, D), generator=gen, device=DEV)) * _weight(D, gen).float()
        s["q"] = q.to(torch.bfloat16)
        s["o"] = torch.zeros((len(Ls), Hq, D), dtype=torch.bfloat16, device=DEV)
    if op == "decode_prefix":
        n = -(-case["prefix"] // PAGE)
        x, _ = _rows(n * PAGE, D, gen, w_k)
        y, _ = _rows(n * PAGE, D, gen)
        s["k_pool"] = torch.cat([s["k_pool"], x.view(n, PAGE, 1, D)])
        s["v_pool"] = torch.cat([s["v_pool"], y.view(n, PAGE, 1, D)])
        s["prefix_table"] = (P + torch.randperm(n, generator=host).to(torch.int32)).to(DEV)
        s["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32, device=DEV)
        s["max_prefix"] = case["prefix"]
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _slots(table, seq, pos):
    return table[seq, pos // PAGE].long() * PAGE + pos % PAGE


def _plain_append(s):
    Hq, Hkv, D = HEADS[s["kind"]]
    theta, pairs = ROPE[s["kind"]]
    T = s["qkv"].shape[0]
    token = torch.arange(T, device=DEV)
    seq = torch.searchsorted(s["cu_q"][1:].long(), token, right=True)
    pos = s["seq_lens"].long()[seq] - s["cu_q"].long()[seq + 1] + token
    x = s["qkv"].float()
    q = _unit(x[:, :Hq * D].view(T, Hq, D)) * s["w_q"].float()
    kv = x[:, Hq * D:].view(T, -1, Hkv, D)
    k = _unit(kv[:, 0]) * s["w_k"].float()
    v = _unit(kv[:, -1])
    freq = theta ** (-2.0 * torch.arange(pairs, device=DEV, dtype=torch.float64) / D)
    angle = pos.double()[:, None, None] * freq  # far positions: in 64 bits
    c, sn = torch.cos(angle).float(), torch.sin(angle).float()
    half = D // 2
    out = []
    for y in (q, k):
        a, b = y[..., :pairs], y[..., half:half + pairs]
        out.append(torch.cat([a * c - b * sn, y[..., pairs:half], b * c + a * sn, y[..., half + pairs:]], -1))
    q, k = out
    s["q_out"].copy_(q)
    slot = _slots(s["table"], seq, pos)
    if s["op"] == "append_chunk":
        s["k_pool"].view(-1, Hkv, D)[slot] = k.to(torch.bfloat16)
        s["v_pool"].view(-1, Hkv, D)[slot] = v.to(torch.bfloat16)
        return s["q_out"], s["k_pool"], s["v_pool"]
    for name, y in (("k", k), ("v", v)):
        z, e = _quantised(y)
        s[name + "_pool"].view(torch.uint8).view(-1, Hkv, D)[slot] = z.view(torch.uint8)
        s[name + "_scale"].view(torch.uint8)[slot // PAGE, :, slot % PAGE] = (e[..., 0] + 127).to(torch.uint8)
    return s["q_out"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"]


def _gather(s, span):
    """The last `span` positions of every sequence (all of the longest one for 0), seen or not: (positions [B, W],
    which exist, slots)."""
    L = s["seq_lens"].long()
    W = min(span, s["max_len"]) if span > 0 else s["max_len"]
    pos = L[:, None] - W + torch.arange(max(W, 1), device=DEV)
    there = pos >= 0
    pos = pos.clamp(min=0)
    seq = torch.arange(L.shape[0], device=DEV)[:, None]
    there = there & (L[:, None] > 0) & (pos < L[:, None])
    return there, _slots(s["table"], seq, pos).clamp(min=0)


def _read(s, name, slot):
    """Cache rows as 32-bit values: [..., Hkv, D]."""
    pool = s[name + "_pool"]
    Hkv, D = pool.shape[2:]
    if pool.dtype == torch.bfloat16:
        return pool.view(-1, Hkv, D)[slot].float()
    x = pool.view(torch.uint8).view(-1, Hkv, D)[slot].view(F8).float()
    e = s[name + "_scale"].view(torch.uint8).transpose(1, 2).reshape(-1, Hkv)[slot]
    return x * torch.exp2(e.float() - 127.0)[..., None]


def _plain_read(s):
    there, slot = _gather(s, s["span"])
    slot = slot[there]
    for name in ("k", "v"):
        out = s[name + "_out"]
        out.view(-1, *out.shape[2:])[slot] = _read(s, name, slot).to(torch.bfloat16)
    return s["k_out"], s["v_out"]


def _scores(s, k):
    """Logits [B, Hkv, G, W] of keys [B, W, Hkv, D]."""
    B, Hq, D = s["q"].shape
    return torch.matmul(s["q"].float().view(B, k.shape[2], -1, D), k.permute(0, 2, 3, 1))


def _softmax_parts(x):
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    return torch.exp(x - m), m


def _plain_decode(s):
    there, slot = _gather(s, WINDOW[s["kind"]])
    x = _scores(s, _read(s, "k", slot)).masked_fill(~there[:, None, None], -math.inf)
    p, _ = _softmax_parts(x)
    o = torch.matmul(p, _read(s, "v", slot).transpose(1, 2)) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    s["o"].copy_(o.view(s["o"].shape))
    return s["o"]


def _plain_prefix(s):
    n = s["max_prefix"]
    pos = torch.arange(n, device=DEV)
    pslot = _slots(s["prefix_table"][None], torch.zeros_like(pos), pos)
    B, Hq, D = s["q"].shape
    there, slot = _gather(s, 0)
    k, v = _read(s, "k", pslot)[:, 0], _read(s, "v", pslot)[:, 0]
    xs = _scores(s, _read(s, "k", slot)).masked_fill(~there[:, None, None], -math.inf)
    x = torch.cat([torch.matmul(s["q"].float().view(B * Hq, D), k.t()).view(B, 1, Hq, n), xs], -1)
    p, _ = _softmax_parts(x)
    o = torch.matmul(p[..., :n].reshape(B * Hq, n), v).view(B, 1, Hq, D)
    o = (o + torch.matmul(p[..., n:], _read(s, "v", slot).transpose(1, 2))) / p.sum(-1, keepdim=True)
    s["o"].copy_(o.view(B, Hq, D))
    return s["o"]


# ---------------------------------------------------------------------------
# the package's calls: prepared once per state, as a serving loop keeps them
# ---------------------------------------------------------------------------

def _prepared(s):
    import paged_decode_attention_gb300 as pda

    kind = s["kind"]
    if s["op"] in ("append_chunk", "append_fp8"):
        name = "chunk" if s["op"] == "append_chunk" else "fp8"
        scales = [] if name == "chunk" else [s["k_scale"], s["v_scale"]]
        fn = getattr(pda, "prepare_kv_append_%s_%s" % (kind, name))
        return fn(s["qkv"], s["w_q"], s["w_k"], s["table"], s["seq_lens"], s["cu_q"], s["k_pool"], s["v_pool"], *scales,
                  q_out=s["q_out"]), tuple(s[n] for n in ("q_out", "k_pool", "v_pool")) + tuple(scales)
    if s["op"] == "read_fp8":
        fn = getattr(pda, "prepare_kv_read_%s_fp8" % kind)
        return fn(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"], s["seq_lens"], s["k_out"],
                  s["v_out"], span=s["span"], max_seq_len=s["max_len"]), (s["k_out"], s["v_out"])
    if s["op"] == "decode_fp8":
        fn = getattr(pda, "prepare_decode_%s_fp8" % kind)
        return fn(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"], s["seq_lens"], s["o"],
                  max_seq_len=s["max_len"]), s["o"]
    return pda.prepare_decode_global_prefix(
        s["q"], s["k_pool"], s["v_pool"], s["prefix_table"], s["prefix_len"], s["table"], s["seq_lens"], s["o"],
        max_prefix_len=s["max_prefix"], max_seq_len=s["max_len"]), s["o"]


def run(state):
    if own:
        if "call" not in state:
            state["call"], state["out"] = _prepared(state)
        state["call"].run(torch.cuda.current_stream())
        return state["out"]
    op = state["op"]
    if op in ("append_chunk", "append_fp8"):
        return _plain_append(state)
    if op == "read_fp8":
        return _plain_read(state)
    return _plain_decode(state) if op == "decode_fp8" else _plain_prefix(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_values():
    """The 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; S.1111.111 is NaN."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        v.append((-x if c & 128 else x) if c & 127 != 127 else math.nan)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _exact_rows(s, name, table, positions, head):
    """Rows of one head at `positions` of a sequence with page list `table`, in 64 bits."""
    page, row = table[positions // PAGE].long(), positions % PAGE
    pool = s[name + "_pool"]
    if pool.dtype == torch.bfloat16:
        return pool[page, row, head].double()
    code = pool.view(torch.uint8)[page, row, head].long()
    scale = s[name + "_scale"].view(torch.uint8)[page, head, row].double()
    return _e4m3_values()[code] * torch.pow(2.0, scale - 127)[:, None]


def _exact_attention(s, case):
    Hq, Hkv, D = HEADS[s["kind"]]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=DEV)
    group = Hq // Hkv
    Ls, _ = _lengths(case)
    for b, L in enumerate(Ls):
        lo = _first(case, L, None)
        pos = torch.arange(lo, L, device=DEV)
        for h in range(Hkv):
            k, v = (_exact_rows(s, n, s["table"][b], pos, h) for n in ("k", "v"))
            if "prefix" in case:
                far = torch.arange(case["prefix"], device=DEV)
                k, v = (torch.cat([_exact_rows(s, n, s["prefix_table"], far, h), x]) for n, x in (("k", k), ("v", v)))
            if k.shape[0]:
                p = torch.softmax(s["q"][b, h * group:(h + 1) * group].double() @ k.t(), -1)
                o[b, h * group:(h + 1) * group] = p @ v
    return o


def _exact_row_norm(x):
    return x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()


def _exact_e4m3(x):
    """Rows rounded to e4m3 at their scales, ties to even: (values, scales)."""
    top = x.abs().max(-1, keepdim=True).values
    k = torch.ceil(torch.log2(top / 448.0)).clamp(-126, 127)
    y = x / torch.pow(2.0, k)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.pow(2.0, e - 3)
    return torch.round(y / step) * step, torch.pow(2.0, k)


def _exact_append(s, case):
    Hq, Hkv, D = HEADS[s["kind"]]
    theta, pairs = ROPE[s["kind"]]
    Ls, new = _lengths(case)
    pos = torch.cat([torch.arange(L - n, L, device=DEV) for L, n in zip(Ls, new)]).double()
    page = torch.cat([s["table"][b][torch.arange(L - n, L, device=DEV) // PAGE] for b, (L, n) in
                      enumerate(zip(Ls, new))]).long()
    row = (pos % PAGE).long()
    x = s["qkv"].double()
    T = x.shape[0]
    i = torch.arange(D // 2, device=DEV).double()
    turn = torch.where(i < pairs, torch.exp(-2.0 * i / D * math.log(theta)), torch.zeros_like(i))
    spin = torch.polar(torch.ones_like(turn)[None, None], pos[:, None, None] * turn)

    def rotated(y):
        z = torch.complex(y[..., :D // 2].contiguous(), y[..., D // 2:].contiguous()) * spin
        return torch.cat([z.real, z.imag], -1)

    q = rotated(_exact_row_norm(x[:, :Hq * D].reshape(T, Hq, D)) * s["w_q"].double())
    src_k = x[:, Hq * D:Hq * D + Hkv * D].reshape(T, Hkv, D)
    src_v = x[:, -Hkv * D:].reshape(T, Hkv, D)
    out = {"k": rotated(_exact_row_norm(src_k) * s["w_k"].double()), "v": _exact_row_norm(src_v)}
    pools, scales = [], []
    for n in ("k", "v"):
        if case["op"] == "append_chunk":
            pool = s[n + "_pool"].double()
            pool[page, row] = out[n]
        else:
            pool = _e4m3_values()[s[n + "_pool"].view(torch.uint8).long()]
            scale = torch.pow(2.0, s[n + "_scale"].view(torch.uint8).double() - 127)
            pool[page, row], k = _exact_e4m3(out[n])
            scale[page, :, row] = k[..., 0]
            scales.append(scale)
        pools.append(pool)
    return tuple([q] + pools + scales)


def _exact_read(s, case):
    Hq, Hkv, D = HEADS[s["kind"]]
    Ls, _ = _lengths(case)
    got = []
    for n in ("k", "v"):
        out = torch.zeros(s[n + "_out"].shape, dtype=torch.float64, device=DEV)
        for b, L in enumerate(Ls):
            pos = torch.arange(_first(case, L, None), L, device=DEV)
            for h in range(Hkv):
                out[s["table"][b][pos // PAGE].long(), pos % PAGE, h] = _exact_rows(s, n, s["table"][b], pos, h)
        got.append(out)
    return tuple(got)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("append_chunk", "append_fp8"):
        return _exact_append(s, case)
    return _exact_read(s, case) if case["op"] == "read_fp8" else _exact_attention(s, case)
