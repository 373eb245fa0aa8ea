"""attn_kv_commit_{sliding,global}: rows moved to the front of their nodes, bit for bit, and nothing else touched."""

import pytest
import torch

import paged_decode_attention_gb300 as pda
from workloads import GLOBAL, PAGE_SIZE, SLIDING

from _tree import DEV, rng

pytestmark = pytest.mark.gpu

SHAPE = {"sliding": SLIDING, "global": GLOBAL}


class Commit:
    def __init__(self, kind, ctx, n, paths, layers=1, seed=0, width=None):
        sh = SHAPE[kind]
        self.kind, self.ctx, self.n, self.paths = kind, ctx, n, paths
        g = torch.Generator().manual_seed(seed)
        L = [c + m for c, m in zip(ctx, n)]
        cols = max(-(-x // PAGE_SIZE) for x in L)
        used = [(b, p) for b, (c, x) in enumerate(zip(ctx, L)) for p in range(c // PAGE_SIZE, -(-x // PAGE_SIZE))]
        P = len(used) + 2
        perm = torch.randperm(P, generator=g).to(torch.int32)
        self.table = torch.full((len(L), max(1, cols)), -1, dtype=torch.int32)
        for i, (b, p) in enumerate(used):
            self.table[b, p] = perm[i]
        shape = (P, PAGE_SIZE, sh["Hkv"], sh["D"])
        self.pools = [torch.randint(-32768, 32767, shape, generator=g, dtype=torch.int16).view(torch.bfloat16)
                      for _ in range(2 * layers)]
        self.lens = torch.tensor(L, dtype=torch.int32)
        cu = [0]
        for m in n:
            cu.append(cu[-1] + m)
        self.cu = torch.tensor(cu, dtype=torch.int32)
        width = max(1, max(len(p) for p in paths)) if width is None else width
        self.path = torch.tensor([p + [-7] * (width - len(p)) for p in paths], dtype=torch.int32)
        self.path_len = torch.tensor([len(p) for p in paths], dtype=torch.int32)

    def rows(self, b, pos):
        pos = torch.tensor(pos, dtype=torch.long)
        return self.table[b][pos // PAGE_SIZE].long(), pos % PAGE_SIZE

    def want(self, skip=()):
        out = [x.clone() for x in self.pools]
        for b, path in enumerate(self.paths):
            if b in skip or not path:
                continue
            src = self.rows(b, [self.ctx[b] + p for p in path])
            dst = self.rows(b, [self.ctx[b] + j for j in range(len(path))])
            for x, old in zip(out, self.pools):
                x[dst] = old[src]
        return out

    def run(self, prepared=False, **kw):
        pools = [x.to(DEV) for x in self.pools]
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        lens = torch.full((len(self.ctx),), -99, dtype=torch.int32, device=DEV)
        args = [pools[0::2], pools[1::2]] + [x.to(DEV) for x in (self.table, self.lens, self.cu, self.path,
                                                                 self.path_len)] + [lens]
        if prepared:
            assert getattr(pda, "prepare_kv_commit_%s" % self.kind)(*args, status=st, **kw).run() is lens
        else:
            assert getattr(pda, "attn_kv_commit_%s" % self.kind)(*args, status=st, **kw) is lens
        torch.cuda.synchronize()
        return [x.cpu() for x in pools], lens.tolist(), int(st.item())


def same(a, b):
    return all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))


def random_commit(kind, layers, seed):
    r = rng(seed)
    n = [r.randint(1, 64) for _ in range(9)] + [0, 64, 64, 1]
    ctx = [r.choice([0, 1, 15, 16, 17, 300]) for _ in n]
    paths = [sorted(r.sample(range(m), r.randint(0, m))) for m in n]
    paths[10], paths[11] = list(range(64)), list(range(40, 64))
    return Commit(kind, ctx, n, paths, layers, seed)


@pytest.mark.parametrize("kind", ["sliding", "global"])
@pytest.mark.parametrize("layers", [1, 3, 64])
def test_paths_of_any_kind(cuda_lib, kind, layers):
    c = random_commit(kind, layers, layers)
    for prepared in (False, True):
        pools, lens, st = c.run(prepared)
        assert st == 0 and same(pools, c.want())
        assert lens == [x + len(p) for x, p in zip(c.ctx, c.paths)]


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_256_sequences(cuda_lib, kind):
    r = rng(4)
    n = [r.randint(1, 12) for _ in range(256)]
    paths = [sorted(r.sample(range(m), r.randint(0, m))) for m in n]
    c = Commit(kind, [r.randint(0, 40) for _ in n], n, paths, 2, 5)
    pools, lens, st = c.run()
    assert st == 0 and same(pools, c.want()) and lens == [x + len(p) for x, p in zip(c.ctx, c.paths)]


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_faults_leave_the_sequence_alone(cuda_lib, kind):
    make = lambda: Commit(kind, [20, 33, 5], [6, 8, 4], [[1, 3, 5], [0, 2, 3, 7], [2]], 2, 7, width=5)  # noqa: E731
    for path, count in (([0, 2, 2, 7], 4), ([3, 2, 5, 7], 4), ([0, 2, 3, 8], 4), ([-1, 2, 3, 7], 4), ([0, 1, 2, 3], -1),
                        ([0, 1, 2, 3], 6), ([0, 1, 2, 3], 2 ** 31 - 1), ([0, 1, 2, 2 ** 31 - 1], 4)):
        c = make()
        c.path[1, :4] = torch.tensor(path, dtype=torch.int32)
        c.path_len[1] = count
        pools, lens, st = c.run()
        assert st == pda.DEV_BAD_TREE and same(pools, c.want(skip=(1,))) and lens == [23, 33, 6]
    for L in (7, -1, 10 ** 6):
        c = make()
        c.lens[1] = L
        pools, lens, st = c.run()
        assert st == pda.DEV_BAD_SEQ_LEN and same(pools, c.want(skip=(1,))) and lens == [23, -99, 6]
    for bad in (-1, 10 ** 6):
        c = make()
        want = c.want(skip=(1,))
        src, dst = c.rows(1, [33 + 2, 33 + 3, 33 + 7]), c.rows(1, [34, 35, 36])
        for x, old in zip(want, c.pools):
            x[dst] = old[src]
        c.table[0, 1] = bad  # rows 20 .. 25 of the first sequence lie there
        want0 = c.want(skip=(0, 1, 2))
        pools, lens, st = c.run()
        page, row = c.rows(2, [5])
        for x, old in zip(want0, c.pools):
            x[dst] = old[src]
            x[page, row] = old[c.rows(2, [7])]
        assert st == pda.DEV_BAD_PAGE and same(pools, want0) and lens == [23, 37, 6]


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_one_pool_each_and_a_new_length_tensor(cuda_lib, kind):
    c = random_commit(kind, 1, 9)
    k, v = (x.to(DEV) for x in c.pools)
    args = [x.to(DEV) for x in (c.table, c.lens, c.cu, c.path, c.path_len)]
    lens = getattr(pda, "attn_kv_commit_%s" % kind)(k, v, *args)
    torch.cuda.synchronize()
    assert same([k.cpu(), v.cpu()], c.want()) and lens.tolist() == [x + len(p) for x, p in zip(c.ctx, c.paths)]
    with pytest.raises(pda.AttnDecodeError, match="twice"):
        getattr(pda, "attn_kv_commit_%s" % kind)([k, k], [v, v], *args)
    with pytest.raises(ValueError):
        getattr(pda, "attn_kv_commit_%s" % kind)([k, k], [v], *args)
