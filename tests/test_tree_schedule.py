"""attn_pages_assign directly in front of attn_decode_*_tree, on a GPU: the attention makes its schedule from the lengths
before it waits for the kernel that writes them, and again where they changed.  Lengths from before the step are other
ones, refused ones or the same; the results and the status have to be those of the step with a synchronize between."""

import pytest
import torch

import paged_decode_attention_gb300 as pda
from workloads import GLOBAL, PAGE_SIZE, SLIDING

from _tree import DEV, random_tree, rng

pytestmark = pytest.mark.gpu

SHAPE = {"sliding": SLIDING, "global": GLOBAL}
CTX = [129, 0, 300, 707, 1, 40]
POOL, ROWS, BLOCKS = 400, 70, 64


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Setting:
    """Six requests with their pages, `leaving` finished ones that give back 200 pages each (a slow assignment), and the
    buffers of a step."""

    def __init__(self, kind, n, leaving, seed):
        sh = SHAPE[kind]
        g = torch.Generator().manual_seed(seed)
        self.kind, self.n, self.B = kind, n, len(CTX) + leaving
        ring, width = 2 * POOL + 200 * leaving, max(BLOCKS, 200)
        ids = torch.randperm(POOL, generator=g).tolist()
        table = torch.full((self.B, width), -1, dtype=torch.int32)
        held = torch.zeros((self.B, 2), dtype=torch.int32)
        for b, c in enumerate(CTX):
            m = -(-c // PAGE_SIZE)
            for p in range(m):
                table[b, p] = ids.pop()
            held[b, 1] = m
        for b in range(len(CTX), self.B):
            table[b, :200] = POOL + torch.arange(200)
            held[b, 1] = 200
        free = torch.full((ring,), -1, dtype=torch.int32)
        head = ring - 5
        free[(head + torch.arange(len(ids))) % ring] = torch.tensor(ids, dtype=torch.int32)
        self.first = [x.to(DEV) for x in (table, held, free)] + [i32([head, len(ids)])]
        self.state = [x.clone() for x in self.first]
        self.cached, self.new = i32(CTX + [0] * leaving), i32(n + [0] * leaving)
        self.lens, self.cu = i32([0] * self.B), i32([0] * (self.B + 1))
        self.q = (torch.randn((ROWS, sh["Hq"], sh["D"]), generator=g) / sh["D"] ** 0.5 * 2.5).to(torch.bfloat16).to(DEV)
        self.k, self.v = (torch.randn((POOL, PAGE_SIZE, sh["Hkv"], sh["D"]), generator=g).to(torch.bfloat16).to(DEV)
                          for _ in "kv")
        r = rng(seed)
        parents = [p for m in n for p in random_tree(m, r)]
        self.parents = i32((parents + [0] * ROWS)[:ROWS])
        self.o = torch.zeros(self.q.shape, dtype=torch.float32, device=DEV)
        self.status = i32([0])

    def assign(self, on):
        on("pages_assign")(self.cached, self.new, *self.state, self.lens, self.cu, status=self.status)

    def attend(self, on, max_q, max_seq_len):
        on("decode_%s_tree" % self.kind)(self.q, self.k, self.v, self.state[0], self.lens, self.cu, self.parents, self.o,
                                         max_q=max_q, max_seq_len=max_seq_len, status=self.status)

    def before(self, lens, cu):
        for x, y in zip(self.state, self.first):
            x.copy_(y)
        self.lens.copy_(i32((lens + [0] * self.B)[:self.B]))
        self.cu.copy_(i32((cu + [cu[-1]] * self.B)[:self.B + 1]))
        self.o.fill_(7.0)
        self.status.zero_()
        torch.cuda.synchronize()

    def after(self):
        torch.cuda.synchronize()
        return [x.clone() for x in (self.o, self.status, self.lens, self.cu, *self.state)]


def stale(n):
    """Lengths of a step before: (seq_lens, cu_q)."""
    cu = [0]
    for m in n:
        cu.append(cu[-1] + m)
    yield [c + m for c, m in zip(CTX, n)], cu            # the same ones
    yield [0] * 6, [0] * 7                               # no tokens
    yield [5, 900, 17, 3, 64, 1], [0, 4, 8, 9, 10, 14, 15]
    yield [1000] * 6, [0, 1, 2, 3, 4, 5, 6]              # more work
    yield [-3, 2 ** 31 - 1, -2 ** 31, 5, 10 ** 6, 1], [0, 3, 1, 2 ** 31 - 1, -2 ** 31, 7, -1]  # refused
    yield [50] * 6, [0, 1, 2, 100, 101, 102, 103]


@pytest.mark.parametrize("mode", ["direct", "graph"])
@pytest.mark.parametrize("leaving", [0, 240])
@pytest.mark.parametrize("kind", ["sliding", "global"])
@pytest.mark.parametrize("n,max_q,max_seq_len", [
    ([4, 2, 0, 3, 1, 4], 4, 730), ([9, 20, 3, 17, 1, 0], 20, 730), ([33, 1, 2, 3, 4, 5], 64, 1024), ([4, 2, 0, 3, 1, 4], 4, 32),
    ([9, 20, 3, 17, 1, 0], 20, 32),
    ([9, 20, 3, 17, 1, 0], 16, 730),   # a sequence of more nodes than the caller's bound: reported, and left alone
    ([30, 20, 3, 27, 1, 0], 64, 730),  # rows past the arrays: the same
])
def test_lengths_written_by_the_kernel_in_front(cuda_lib, kind, n, max_q, max_seq_len, leaving, mode):
    s = Setting(kind, n, leaving, seed=max_q + leaving)
    s.before([0], [0])
    one = lambda name: getattr(pda, "attn_" + name)  # noqa: E731
    s.assign(one)
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0 and s.cu.tolist()[6] == sum(n)
    s.attend(one, max_q, max_seq_len)
    want = s.after()
    fits = max(n) <= max_q and sum(n) <= ROWS
    assert int(want[1].item()) == (0 if fits else pda.DEV_BAD_SEQ_LEN)
    at = 0
    for m in n:
        left = m > max_q or at + m > ROWS
        rows = want[0][at:min(at + m, ROWS)]
        assert (rows == 7.0).all() if left else torch.isfinite(rows).all() and not (rows == 7.0).all(-1).any()
        at += m
    step = pda.Step()
    on = lambda name: getattr(step, "add_" + name)  # noqa: E731
    s.assign(on)
    s.attend(on, max_q, max_seq_len)
    step.finalize(mode)
    for lens, cu in stale(n):
        for _ in range(3):
            s.before(lens, cu)
            step.launch()
            assert all(torch.equal(a, b) for a, b in zip(s.after(), want)), (lens, cu)
    step.close()
