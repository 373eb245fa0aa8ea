"""Verification steps as a server runs them: pages assigned, trees appended and attended to, paths committed, on both layer
types over one another's steps.  The cache has to hold, bit for bit, what appending the accepted text at once gives, and
every node has to see exactly its text."""

import pytest
import torch

import paged_decode_attention_gb300 as pda
from workloads import GLOBAL, PAGE_SIZE, SLIDING, append_row_len

from _fp8 import decode_bound
from _tree import DEV, chains_of, random_tree, rng

pytestmark = pytest.mark.gpu

SHAPE = {"sliding": SLIDING, "global": GLOBAL}
B, ROWS, BLOCKS, MAX_N = 3, 150, 20, 24
WINDOW = {"sliding": 40, "global": 0}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Layer:
    """One layer's state and buffers; the same ones in every step."""

    def __init__(self, kind, seed, pages):
        self.kind, self.window = kind, WINDOW[kind]
        sh = SHAPE[kind]
        g = torch.Generator().manual_seed(seed)
        self.Hq, self.Hkv, self.D = sh["Hq"], sh["Hkv"], sh["D"]
        self.w_q, self.w_k = ((0.3 * (1 + 0.1 * torch.randn(self.D, generator=g))).to(torch.bfloat16).to(DEV) for _ in "qk")
        self.qkv = torch.zeros((ROWS, append_row_len(kind)), dtype=torch.bfloat16, device=DEV)
        self.k, self.v = (torch.full((pages, PAGE_SIZE, self.Hkv, self.D), float("nan"), dtype=torch.bfloat16, device=DEV)
                          for _ in "kv")
        self.state = pda.new_page_state(pages, B, BLOCKS, DEV)
        self.seq_lens, self.cu = i32([0] * B), i32([0] * (B + 1))
        self.q = torch.zeros((ROWS, self.Hq, self.D), dtype=torch.bfloat16, device=DEV)
        self.o = torch.zeros((ROWS, self.Hq, self.D), dtype=torch.float32, device=DEV)
        self.texts = [torch.zeros((0, self.qkv.shape[1]), dtype=torch.bfloat16) for _ in range(B)]

    def appended(self, rows):
        """(q, k, v) of a text appended at once into a cache of its own."""
        n = rows.shape[0]
        blocks = max(1, -(-n // PAGE_SIZE))
        k, v = (torch.zeros((blocks, PAGE_SIZE, self.Hkv, self.D), dtype=torch.bfloat16, device=DEV) for _ in "kv")
        table = torch.arange(blocks, dtype=torch.int32, device=DEV)[None]
        q = getattr(pda, "attn_kv_append_%s_chunk" % self.kind)(rows.to(DEV), self.w_q, self.w_k, table, i32([n]),
                                                                i32([0, n]), k, v)
        return q, k.view(-1, self.Hkv, self.D)[:n], v.view(-1, self.Hkv, self.D)[:n]


def attend(layer, q, k, v):
    """The last position's attention in 64 bits: (o, A, S) [Hq, D], [Hq, D], [Hq, 1]."""
    lo = max(0, k.shape[0] - layer.window) if layer.window > 0 else 0
    k, v, q = k[lo:].double(), v[lo:].double(), q[-1].double()
    G = layer.Hq // layer.Hkv
    k, v = k.repeat_interleave(G, 1).transpose(0, 1), v.repeat_interleave(G, 1).transpose(0, 1)
    x = torch.einsum("hd,hld->hl", q, k)
    w = torch.softmax(x, -1)
    S = torch.einsum("hd,hld->hl", q.abs(), k.abs()).amax(-1, keepdim=True)
    return torch.einsum("hl,hld->hd", w, v), torch.einsum("hl,hld->hd", w, v.abs()), S


@pytest.mark.parametrize("mode", ["calls", "direct", "graph"])
def test_a_run_of_steps(cuda_lib, mode):
    r = rng(17)
    g = torch.Generator().manual_seed(18)
    layers = [Layer("sliding", 1, 30), Layer("global", 2, 60)]
    cached, new, parents = i32([0] * B), i32([0] * B), i32([-1] * ROWS)
    path, path_len, new_lens = i32([[0] * MAX_N] * B), i32([0] * B), i32([0] * B)
    status = i32([0])
    steps = []

    def calls(on):
        for x in layers:
            on("pages_assign")(cached, new, *x.state, x.seq_lens, x.cu, window=x.window, status=status)
            on("kv_append_%s_tree" % x.kind)(x.qkv, x.w_q, x.w_k, x.state[0], x.seq_lens, x.cu, parents, x.k, x.v, x.q,
                                             status=status)
            on("decode_%s_tree" % x.kind)(x.q, x.k, x.v, x.state[0], x.seq_lens, x.cu, parents, x.o, max_q=MAX_N,
                                          max_seq_len=BLOCKS * PAGE_SIZE, window=x.window, status=status)

    def commits(on):
        for x in layers:
            on("kv_commit_%s" % x.kind)([x.k], [x.v], x.state[0], x.seq_lens, x.cu, path, path_len, new_lens,
                                        status=status)

    if mode != "calls":
        for record in (calls, commits):
            step = pda.Step()
            record(lambda name: getattr(step, "add_" + name))
            steps.append(step.finalize(mode))
            assert step.launch_mode == mode

    for turn in range(9):
        # a prompt first (chains), then trees; one request ends in the middle and another takes its row
        if turn == 5:
            for x in layers:
                x.texts[1] = x.texts[1][:0]
        trees = []
        for b in range(B):
            fresh = layers[0].texts[b].shape[0] == 0
            n = r.randint(5, MAX_N) if fresh else r.choice([1, 2, 7, MAX_N, 0 if turn > 2 else 3])
            trees.append([i - 1 for i in range(n)] if fresh else random_tree(n, r, roots=0.0))
        cached.copy_(i32([layers[0].texts[b].shape[0] for b in range(B)]))
        new.copy_(i32([len(t) for t in trees]))
        flat = [p for t in trees for p in t]
        parents[:len(flat)] = i32(flat)
        rows = {}
        for x in layers:
            rows[x.kind] = torch.randn((len(flat), x.qkv.shape[1]), generator=g).to(torch.bfloat16)
            x.qkv[:len(flat)] = rows[x.kind].to(DEV)
            x.o.fill_(7.0)
        torch.cuda.synchronize()
        if mode == "calls":
            calls(lambda name: getattr(pda, "attn_" + name))
        else:
            steps[0].launch()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        chains = [chains_of(t) for t in trees]
        for x in layers:
            assert (x.o[len(flat):] == 7.0).all()
            at = 0
            for b in range(B):
                for i in {0, len(trees[b]) // 2, len(trees[b]) - 1} if trees[b] else ():
                    text = torch.cat([x.texts[b], rows[x.kind][at:at + len(trees[b])][chains[b][i]]])
                    q, k, v = x.appended(text)
                    o, A, S = attend(x, q, k, v)
                    assert torch.equal(x.q[at + i], q[-1])
                    bound = decode_bound(o, A, S, x.D, torch.float32, 2.0 ** -8)
                    assert ((x.o[at + i].double() - o).abs() <= bound).all()
                at += len(trees[b])
        # the accepted path: all of a prompt, some chain of a tree
        taken = []
        for b in range(B):
            fresh = layers[0].texts[b].shape[0] == 0
            chain = chains[b][-1 if fresh else r.randrange(len(chains[b]))] if chains[b] else []
            taken.append(chain)
            path[b, :len(chain)] = i32(chain) if chain else path[b, :0]
        path_len.copy_(i32([len(c) for c in taken]))
        torch.cuda.synchronize()
        if mode == "calls":
            commits(lambda name: getattr(pda, "attn_" + name))
        else:
            steps[1].launch()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        for x in layers:
            at = 0
            for b in range(B):
                x.texts[b] = torch.cat([x.texts[b], rows[x.kind][at:at + len(trees[b])][taken[b]]])
                at += len(trees[b])
                n = x.texts[b].shape[0]
                assert int(new_lens[b]) == n
                if n == 0:
                    continue
                _, k, v = x.appended(x.texts[b])
                lo = max(0, n - x.window + 1) if x.window > 0 else 0
                pos = torch.arange(lo, n, device=DEV)
                page, row = x.state[0][b][pos // PAGE_SIZE].long(), pos % PAGE_SIZE
                assert torch.equal(x.k[page, row], k[lo:]) and torch.equal(x.v[page, row], v[lo:])
    for s in steps:
        s.close()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_calls_on_another_stream_order_their_own_memory(cuda_lib, kind):
    """Outputs and workspaces that a call makes for itself, with the default stream held back by slow kernels."""
    from _tree import TreeCase, chain
    c = TreeCase(kind, [900, 40], [chain(6), chain(9)], seed=3, fill=0.0)
    kw = dict(window=c.window, max_q=9, max_seq_len=906, out_dtype=torch.float32)
    fn = getattr(pda, "attn_decode_%s_tree" % kind)
    args = c.args()
    want = fn(*args, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for held in (torch.cuda.current_stream(), side):
        for _ in range(3):
            with torch.cuda.stream(held):
                torch.cuda._sleep(2_000_000)
            got = fn(*args, stream=side, **kw)
            junk = [torch.full((1 << 18,), 3.0, device=DEV) for _ in range(4)]  # would take the call's memory
            side.synchronize()
            assert torch.equal(got, want)
            del junk
    call = getattr(pda, "prepare_decode_%s_tree" % kind)(*args, **kw)
    out = call.run(side)
    side.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_the_step_s_other_calls_on_another_stream(cuda_lib, kind):
    """The append's rows, the commit's lengths and the page tables, each made by its call, one stream held back."""
    _, Hkv, D = pda.SHAPES[getattr(pda, "KIND_" + kind.upper())]
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn((12, append_row_len(kind)), generator=g).to(torch.bfloat16).to(DEV)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    parents, path = i32([-1, 0, 0, 2, -1, 0, 1, 2, 3, 4, 5, 6]), i32([[1, 3, 0], [0, 2, 7]])
    cached, new, path_len = i32([30, 5]), i32([4, 8]), i32([2, 3])
    pool = torch.randn((9, PAGE_SIZE, Hkv, D), generator=g).to(torch.bfloat16).to(DEV)
    call = lambda name: getattr(pda, name % kind)  # noqa: E731

    def run(stream):
        kw = dict(stream=stream)
        with torch.cuda.stream(stream):
            state = pda.new_page_state(9, 2, 3, DEV)
            pools = [pool.clone() for _ in range(4)]
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
        stream.synchronize()
        with torch.cuda.stream(side if stream != side else torch.cuda.default_stream()):
            torch.cuda._sleep(2_000_000)
        lens, cu = pda.attn_pages_assign(cached, new, *state, status=status, **kw)
        q = call("attn_kv_append_%s_tree")(qkv, w, w, state[0], lens, cu, parents, *pools[:2], status=status, **kw)
        kept = call("attn_kv_commit_%s")(pools[0::2], pools[1::2], state[0], lens, cu, path, path_len, status=status, **kw)
        junk = [torch.full((1 << 12,), 3.0, device=DEV) for _ in range(8)]  # would take the calls' memory
        stream.synchronize()
        assert int(status.item()) == 0 and kept.tolist() == [32, 8] and len(junk) == 8
        torch.cuda.synchronize()
        return [lens, cu, q, kept, *state, *pools]

    side = torch.cuda.Stream()
    want = run(torch.cuda.default_stream())
    for stream in (side, torch.cuda.default_stream(), side):
        assert all(torch.equal(a, b) for a, b in zip(run(stream), want))


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_two_graphs_of_one_workspace_replayed_in_turn(cuda_lib, kind):
    """Calls of other sizes behind one another in one workspace, each captured; nothing is kept in it between them."""
    from _tree import TreeCase, chain, random_tree
    cases = [TreeCase(kind, [900, 40, 3000], [chain(6), chain(9), random_tree(40, rng(1))], seed=3, fill=0.0),
             TreeCase(kind, [5000], [random_tree(5, rng(2))], seed=4, fill=0.0)]
    ws = torch.full((1 << 28,), 255, dtype=torch.uint8, device=DEV)  # (NaN, and cuts that name no rows)
    graphs, calls, want = [], [], []
    for c in cases:
        kw = dict(window=c.window, max_q=c.max_n, max_seq_len=max(c.L), out_dtype=torch.float32)
        want.append(getattr(pda, "attn_decode_%s_tree" % kind)(*c.args(), **kw))
        calls.append(getattr(pda, "prepare_decode_%s_tree" % kind)(*c.args(), workspace=ws, **kw))
        calls[-1].run()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            calls[-1].run()
    for order in ((0, 1), (1, 0), (0, 0, 1, 1, 0)):
        for call in calls:
            call.out.fill_(7.0)
        torch.cuda.synchronize()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(call.out, w) for call, w in zip(calls, want))


def test_pages_beyond_32_bit_offsets(cuda_lib):
    """The last pages of a pool of more than 2^31 elements, against the same pages in a small one."""
    from _tree import TreeCase, chain
    c = TreeCase("sliding", [900, 40], [random_tree(30, rng(3)), chain(9)], seed=3, fill=0.0)
    q, k, v, table, lens, cu, parents = c.args()
    n, P = 70000, k.shape[0]
    g = torch.Generator().manual_seed(8)
    qkv = torch.randn((39, append_row_len("sliding")), generator=g).to(torch.bfloat16).to(DEV)
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    path, path_len = i32([list(range(1, 30, 3)), list(range(10))]), i32([10, 9])
    results = []
    for off in (0, n - P):
        pools = [k.clone(), v.clone()] if off == 0 else [torch.empty((n,) + k.shape[1:], dtype=k.dtype, device=DEV)
                                                         for _ in "kv"]
        if off:
            pools[0][off:], pools[1][off:] = k, v
        at = torch.where(table >= 0, table + off, table).to(torch.int32)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = [pda.attn_kv_append_sliding_tree(qkv, w, w, at, lens, cu, parents, *pools, status=status)]
        out.append(pda.attn_decode_sliding_tree(q, *pools, at, lens, cu, parents, status=status))
        out.append(pda.attn_kv_commit_sliding(*pools, at, lens, cu, path, path_len, status=status))
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        results.append(out + [x[off:].clone() for x in pools])
    assert all(torch.equal(a, b) for a, b in zip(*results))
