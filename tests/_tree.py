"""Trees of drafted tokens for the tests: cases over a paged cache, and the attention's definition in 64 bits."""

import random

import torch

from workloads import GLOBAL, PAGE_SIZE, SLIDING

DEV = "cuda:0"
SHAPE = {"sliding": SLIDING, "global": GLOBAL}


def random_tree(n, rng, roots=0.05):
    """Parents of n nodes: any earlier node, now and then the context itself."""
    return [-1 if i == 0 or rng.random() < roots else rng.randrange(i) for i in range(n)]


def chain(n):
    return [i - 1 for i in range(n)]


def star(n):
    return [-1] * min(n, 1) + [0] * (n - 1)


def chains_of(parents):
    """Every node's ancestors, itself last; a parent outside [-1, i) counts as -1."""
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if 0 <= p < i else []) + [i])
    return out


class TreeCase:
    """ctx[b] cached tokens and a tree trees[b] per sequence.  Pool rows that no node sees hold `fill`."""

    def __init__(self, kind, ctx, trees, seed, window=None, spare=0, scale=1.0, fill=float("nan"), extra_pages=2):
        sh = SHAPE[kind]
        self.kind, self.ctx, self.trees = kind, list(ctx), [list(t) for t in trees]
        self.Hq, self.Hkv, self.D = sh["Hq"], sh["Hkv"], sh["D"]
        self.window = (1024 if kind == "sliding" else 0) if window is None else window
        g = torch.Generator().manual_seed(seed)
        self.n = [len(t) for t in self.trees]
        self.L = [c + n for c, n in zip(self.ctx, self.n)]
        self.T = sum(self.n)
        self.lo = [max(0, c - self.window + 1) if self.window > 0 else 0 for c in self.ctx]
        width = max(1, max((-(-x // PAGE_SIZE) for x in self.L), default=1))
        need = [(b, p) for b in range(len(self.L)) if self.n[b]
                for p in range(self.lo[b] // PAGE_SIZE, -(-self.L[b] // PAGE_SIZE))]
        self.P = len(need) + extra_pages
        perm = torch.randperm(self.P, generator=g).to(torch.int32)
        self.table = torch.full((len(self.L), width), -1, dtype=torch.int32)
        for i, (b, p) in enumerate(need):
            self.table[b, p] = perm[i]
        shape = (self.P, PAGE_SIZE, self.Hkv, self.D)
        self.k = torch.full(shape, fill, dtype=torch.bfloat16)
        self.v = torch.full(shape, fill, dtype=torch.bfloat16)
        for b in range(len(self.L)):
            if self.n[b]:
                page, row = self.slot(b, torch.arange(self.lo[b], self.L[b]))
                m = page.shape[0]
                self.k[page, row] = torch.randn((m, self.Hkv, self.D), generator=g).to(torch.bfloat16)
                self.v[page, row] = torch.randn((m, self.Hkv, self.D), generator=g).to(torch.bfloat16)
        self.q = (scale * torch.randn((self.T + spare, self.Hq, self.D), generator=g) / self.D ** 0.5 * 2.5).to(
            torch.bfloat16)
        self.parents = torch.tensor([p for t in self.trees for p in t] + [0] * spare, dtype=torch.int32)
        cu = [0]
        for n in self.n:
            cu.append(cu[-1] + n)
        self.cu = torch.tensor(cu, dtype=torch.int32)
        self.lens = torch.tensor(self.L, dtype=torch.int32)
        self.max_n = max(self.n)

    def slot(self, b, positions):
        return self.table[b][positions // PAGE_SIZE].long(), positions % PAGE_SIZE

    def args(self):
        return [x.to(DEV) for x in (self.q, self.k, self.v, self.table, self.lens, self.cu, self.parents)]

    def seen(self, b):
        """[n, L - lo] what every node of sequence b sees, from position lo on."""
        c, n, lo, w = self.ctx[b], self.n[b], self.lo[b], self.window
        chains = chains_of(self.trees[b])
        m = torch.zeros((n, c + n - lo), dtype=torch.bool)
        for i, up in enumerate(chains):
            here = c + len(up) - 1
            m[i, max(0, (here - w + 1 if w > 0 else 0) - lo):c - lo] = True
            for a in up:
                if w <= 0 or len(up) - len(chains[a]) < w:
                    m[i, c - lo + a] = True
        return m

    def want(self):
        """(o, A, S) [T, Hq, D] and [T, Hq, 1] in 64 bits: the outputs, sum w |v| / sum w, and the largest sum |q_i k_i|."""
        o = torch.zeros((self.T, self.Hq, self.D), dtype=torch.float64)
        A, S = torch.zeros_like(o), torch.zeros((self.T, self.Hq, 1), dtype=torch.float64)
        G, at = self.Hq // self.Hkv, 0
        for b in range(len(self.L)):
            n = self.n[b]
            if n == 0:
                continue
            seen = self.seen(b)
            page, row = self.slot(b, torch.arange(self.lo[b], self.L[b]))
            for h in range(self.Hkv):
                k, v = self.k[page, row, h].double(), self.v[page, row, h].double()
                for g in range(G):
                    q = self.q[at:at + n, h * G + g].double()
                    w = torch.softmax((q @ k.t()).masked_fill(~seen, float("-inf")), -1)
                    o[at:at + n, h * G + g] = w @ v
                    A[at:at + n, h * G + g] = w @ v.abs()
                    S[at:at + n, h * G + g, 0] = (q.abs() @ k.abs().t()).masked_fill(~seen, 0).max(-1).values
            at += n
        return o, A, S


def run_tree(pda, c, out_dtype=torch.float32, prepared=False, fill=7.0, **kw):
    """(o of every row, status): o holds `fill` where the call writes nothing."""
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    o = torch.full(c.q.shape, fill, dtype=out_dtype, device=DEV)
    kw = dict(dict(window=c.window, max_q=c.max_n, max_seq_len=max(c.L), status=st), **kw)
    args = c.args() + [o]
    if prepared:
        call = getattr(pda, "prepare_decode_%s_tree" % c.kind)(*args, **kw)
        assert call.run() is o
    else:
        assert getattr(pda, "attn_decode_%s_tree" % c.kind)(*args, **kw) is o
    torch.cuda.synchronize()
    return o, int(st.item())


def rng(seed):
    return random.Random(seed)
