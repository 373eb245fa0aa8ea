"""attn_pages_assign against a list model of the same free list, step after step."""

import pytest
import torch

import paged_decode_attention_gb300 as pda

from _tree import DEV, rng

pytestmark = pytest.mark.gpu


class Model:
    """What the call does, in Python lists."""

    def __init__(self, pages, batch, blocks, window=0):
        self.pages, self.blocks, self.window = pages, blocks, window
        self.table = [[-1] * blocks for _ in range(batch)]
        self.held = [[0, 0] for _ in range(batch)]
        self.free, self.head = list(range(pages)), 0

    def range(self, cached, new):
        first = max(0, cached - self.window + 1) // 16 if self.window > 0 else 0
        return [first, max(first, -(-(cached + new) // 16))]

    def step(self, cached, new):
        """None, or the fault's status bit."""
        ranges = []
        for b, (c, n) in enumerate(zip(cached, new)):
            if c < 0 or n < 0 or c + n > min(self.blocks * 16, 262144):
                return pda.DEV_BAD_SEQ_LEN
            ranges.append(self.range(c, n))
            if self.held[b][0] < self.held[b][1] and ranges[b][0] < self.held[b][0] and c > 0:
                return pda.DEV_BAD_SEQ_LEN
        take = [(b, p) for b, r in enumerate(ranges) for p in range(*r) if not self.held[b][0] <= p < self.held[b][1]]
        give = [(b, p) for b, h in enumerate(self.held) for p in range(*h) if not ranges[b][0] <= p < ranges[b][1]]
        if len(take) > len(self.free):
            return pda.DEV_NO_PAGES
        got, self.free = self.free[:len(take)], self.free[len(take):]
        self.free += [self.table[b][p] for b, p in give]
        self.head = (self.head + len(take)) % self.pages
        for (b, p), page in zip(take, got):
            self.table[b][p] = page
        self.held = ranges
        return None


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Device:
    def __init__(self, m, batch):
        self.m = m
        self.state = pda.new_page_state(m.pages, batch, m.blocks, DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step(self, cached, new, **kw):
        lens, cu = pda.attn_pages_assign(i32(cached), i32(new), *self.state, window=self.m.window, status=self.status, **kw)
        torch.cuda.synchronize()
        return lens.tolist(), cu.tolist()

    def check(self):
        table, held, free, state = (x.tolist() for x in self.state)
        assert table == self.m.table and held == self.m.held and state == [self.m.head, len(self.m.free)]
        assert [free[(self.m.head + i) % self.m.pages] for i in range(len(self.m.free))] == self.m.free
        used = [table[b][p] for b, h in enumerate(held) for p in range(*h)]
        assert sorted(used + self.m.free) == list(range(self.m.pages))


def cumulative(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


@pytest.mark.parametrize("window", [0, 40, 1024])
@pytest.mark.parametrize("batch,blocks,pages", [(1, 30, 40), (7, 200, 900), (64, 90, 5000), (256, 130, 30000), (33, 1, 33)])
def test_steps_of_a_running_batch(cuda_lib, window, batch, blocks, pages):
    r = rng(batch + window)
    m = Model(pages, batch, blocks, window)
    d = Device(m, batch)
    cached = [0] * batch
    refused = 0
    for step in range(25):
        new = []
        for b in range(batch):
            u = r.random()
            if u < 0.08:  # finished, or another request in its place
                cached[b] = 0
                new.append(0 if r.random() < 0.5 else r.randint(0, blocks * 16))
            elif u < 0.2:
                new.append(0)
            else:
                new.append(min(r.randint(1, 64), blocks * 16 - cached[b]))
        fault = m.step(cached, new)
        lens, cu = d.step(cached, new)
        if fault is None:
            assert int(d.status.item()) == 0
            assert lens == [c + n for c, n in zip(cached, new)] and cu == cumulative(new)
            cached = [c + r.randint(0, n) for c, n in zip(cached, new)]  # what was accepted
        else:
            refused += 1
            assert int(d.status.item()) == fault
            d.status.zero_()
            assert lens == cached and cu == [0] * (batch + 1)
        d.check()
    assert refused < 20


def test_faults_change_nothing(cuda_lib):
    m = Model(20, 3, 12, 32)
    d = Device(m, 3)
    for cached, new in (([0, 0, 0], [100, 30, 0]), ([90, 30, 0], [20, 1, 5])):
        assert m.step(cached, new) is None
        d.step(cached, new)
        d.check()
    for cached, new, bit, lens in (
            ([90, -1, 0], [1, 1, 1], pda.DEV_BAD_SEQ_LEN, [90, 0, 0]),
            ([90, 30, 0], [1, -2, 1], pda.DEV_BAD_SEQ_LEN, [90, 30, 0]),
            ([90, 30, 0], [103, 1, 1], pda.DEV_BAD_SEQ_LEN, [90, 30, 0]),
            ([90, 30, 2 ** 31 - 1], [1, 1, 2 ** 31 - 1], pda.DEV_BAD_SEQ_LEN, [90, 30, 192]),
            ([20, 30, 0], [1, 1, 1], pda.DEV_BAD_SEQ_LEN, [20, 30, 0]),  # its first pages were given back
            ([90, 30, 0], [100, 160, 190], pda.DEV_NO_PAGES, [90, 30, 0])):
        got, cu = d.step(cached, new)
        assert int(d.status.item()) == bit and got == lens and cu == [0] * 4
        d.status.zero_()
        d.check()
    for state in ([-1, 3], [20, 3], [0, -1], [0, 21], [0, 20]):  # a free list whose numbers do not fit
        keep = d.state[3].clone()
        d.state[3].copy_(i32(state))
        _, cu = d.step([0, 0, 0], [0, 0, 0])
        assert int(d.status.item()) == pda.DEV_BAD_SEQ_LEN and cu == [0] * 4 and d.state[3].tolist() == state
        d.state[3].copy_(keep)
        d.status.zero_()
        d.check()
    for held in ([-1, 4], [5, 4], [0, 13]):
        keep = d.state[1].clone()
        d.state[1][1] = i32(held)
        d.step([90, 30, 0], [1, 1, 1])
        assert int(d.status.item()) == pda.DEV_BAD_SEQ_LEN
        d.state[1].copy_(keep)
        d.status.zero_()
        d.check()


def test_the_state_may_go_elsewhere_and_steps_replay(cuda_lib):
    m = Model(64, 4, 20)
    d = Device(m, 4)
    held, state = torch.empty_like(d.state[1]), torch.empty_like(d.state[3])
    before = [x.clone() for x in (d.state[1], d.state[3])]
    for _ in range(2):  # from the same state twice: the same answer
        lens, cu = d.step([0] * 4, [20, 0, 17, 300], held_out=held, free_state_out=state)
        assert int(d.status.item()) == 0 and lens == [20, 0, 17, 300] and cu == [0, 20, 20, 37, 337]
        assert all(torch.equal(x, y) for x, y in zip((d.state[1], d.state[3]), before))
    assert m.step([0] * 4, [20, 0, 17, 300]) is None
    d.state[1].copy_(held)
    d.state[3].copy_(state)
    d.check()
    # captured: lengths change between replays, the state moves on in place
    cached, new = i32([20, 0, 17, 300]), i32([1, 1, 1, 1])
    call = pda.prepare_pages_assign(cached, new, *d.state, status=d.status)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call.run()
    for c, n in (([20, 0, 17, 300], [1, 64, 16, 20]), ([21, 40, 17, 0], [15, 0, 16, 0]), ([0, 41, 33, 0], [0, 7, 64, 5])):
        cached.copy_(i32(c))
        new.copy_(i32(n))
        graph.replay()
        torch.cuda.synchronize()
        assert m.step(c, n) is None and int(d.status.item()) == 0
        assert call.out[0].tolist() == [x + y for x, y in zip(c, n)] and call.out[1].tolist() == cumulative(n)
        d.check()
