"""Decode behind a shared prefix (attn_decode_global_prefix) against the definition in 64 bits, element by element within
_fp8.decode_bound for bf16 weights.  Every slot that no query may read is NaN."""

import numpy as np
import pytest
import torch

import paged_decode_attention_gb300 as pda
from workloads import append_row_len, make_case

from _fp8 import attention_rows, decode_bound

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
WEIGHT_EPS = torch.finfo(torch.bfloat16).eps / 2


class Case:
    def __init__(self, prefix, lens, seed, q_scale=1.0, spare_blocks=0):
        own = make_case("global", lens, seed)
        pre = make_case("global", [prefix], seed + 1)
        P = own.num_pages
        self.q = (own.q.float() * q_scale).to(torch.bfloat16)
        self.k = torch.cat([own.k_pool, pre.k_pool])
        self.v = torch.cat([own.v_pool, pre.v_pool])
        t = pre.block_table[0]
        self.prefix_table = torch.cat([torch.where(t >= 0, t + P, t), torch.full((spare_blocks,), -1)]).to(torch.int32)
        self.prefix = prefix
        self.table, self.lens = own.block_table, lens

    def args(self):
        return [x.to(DEV) for x in (self.q, self.k, self.v, self.prefix_table,
                                    torch.tensor([self.prefix], dtype=torch.int32), self.table,
                                    torch.tensor(self.lens, dtype=torch.int32))]


# prefix_splits=0 takes one list of pages per sequence for small cases; the cases below run both ways
BOTH = pytest.mark.parametrize("splits", [0, 2])


def decode(args, **kw):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw.setdefault("out_dtype", torch.float32)
    o = pda.attn_decode_global_prefix(*args, status=st, **kw)
    torch.cuda.synchronize()
    return o, int(st.item())


def check(c, label="", **kw):
    args = c.args()
    o, st = decode(args, **kw)
    assert st == 0, "%s: status %d" % (label, st)
    q, k, v, pt, _, bt, sl = args
    want, A, S = attention_rows(q, k, v, bt, sl, 0, prefix=(pt, c.prefix))
    bound = decode_bound(want, A, S, 512, o.dtype, WEIGHT_EPS)
    got = o.double().cpu()
    assert torch.isfinite(got).all(), label
    err = (got - want).abs()
    assert (err <= bound).all(), "%s: %.3g times the bound" % (label, float((err / bound).max()))
    return o


@BOTH
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 63, 64, 65, 255, 257, 1000, 1024])
def test_prefix_lengths(cuda_lib, prefix, splits):
    check(Case(prefix, [0, 1, 17, 300, 64], seed=61, spare_blocks=2), "prefix %d" % prefix, prefix_splits=splits)


@BOTH
@pytest.mark.parametrize("batch", [1, 7, 8, 9, 15, 16, 17, 33, 100])
def test_batches(cuda_lib, batch, splits):
    r = np.random.RandomState(batch)
    check(Case(700, r.randint(0, 60, batch).tolist(), seed=62), prefix_splits=splits)


def test_full_batch(cuda_lib):
    r = np.random.RandomState(3)
    check(Case(131, r.randint(0, 30, 256).tolist(), seed=63))


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_a_long_prefix(cuda_lib, out_dtype):
    check(Case(9001, [0, 5, 1500, 33, 16, 1, 0, 700, 80], seed=64), out_dtype=out_dtype)


@pytest.mark.parametrize("num_splits", [0, 2])
@pytest.mark.parametrize("prefix,lens", [(0, [0, 3]), (1, [0, 0]), (17, [0, 30, 1]), (16, [48]),
                                         (50, [r % 60 for r in range(20)])])
def test_short_lists_whole_and_cut(cuda_lib, prefix, lens, num_splits):
    check(Case(prefix, lens, seed=78), num_splits=num_splits)


@BOTH
@pytest.mark.parametrize("prefix,lens", [(20001, [0]), (9000, [700]), (15, [16000]), (8192, [0, 33])])
def test_one_or_two_sequences_in_many_partials(cuda_lib, prefix, lens, splits):
    check(Case(prefix, lens, seed=77), prefix_splits=splits)


@pytest.mark.parametrize("prefix_splits", [0, 1, 2, 3, 16, 128, 1000])
@pytest.mark.parametrize("num_splits", [0, 1, 50])
def test_forced_splits(cuda_lib, num_splits, prefix_splits):
    check(Case(1300, [3, 0, 600, 1100], seed=65), num_splits=num_splits, prefix_splits=prefix_splits)


@BOTH
def test_nothing_visible_gives_zero(cuda_lib, splits):
    c = Case(0, [0, 40, 0], seed=66)
    o = check(c, prefix_splits=splits)
    assert (o[0] == 0).all() and (o[2] == 0).all()


@BOTH
@pytest.mark.parametrize("q_scale", [0.0, 0.05, 8.0])
def test_flat_and_dominated_weights(cuda_lib, q_scale, splits):
    check(Case(900, [5, 0, 1200], seed=67, q_scale=q_scale), prefix_splits=splits)


@BOTH
def test_bounds_size_the_launches_only(cuda_lib, splits):
    c = Case(1000, [5, 0, 700, 33], seed=68)
    args = c.args()
    o, st = decode(args, prefix_splits=splits)
    assert st == 0
    want, A, S = attention_rows(args[0], args[1], args[2], args[5], args[6], 0, prefix=(args[3], c.prefix))
    for bounds in (dict(max_prefix_len=0, max_seq_len=0), dict(max_prefix_len=16, max_seq_len=700)):
        o, st = decode(args, prefix_splits=splits, **bounds)
        assert st == 0
        assert ((o.double().cpu() - want).abs() <= decode_bound(want, A, S, 512, o.dtype, WEIGHT_EPS)).all()


@BOTH
def test_whole_pages_equal_the_plain_decode_over_joined_tables(cuda_lib, splits):
    c = Case(640, [5, 17, 700], seed=69)
    q, k, v, pt, _, bt, sl = c.args()
    o, _ = decode(c.args(), prefix_splits=splits)
    joined = torch.cat([pt[None].expand(3, -1), bt], 1).contiguous()
    plain = pda.attn_decode_global(q, k, v, joined, sl + 640, out_dtype=torch.float32)
    torch.cuda.synchronize()
    want, A, S = attention_rows(q, k, v, joined, sl + 640, 0)
    bound = decode_bound(want, A, S, 512, torch.float32, WEIGHT_EPS)
    assert ((o - plain).abs().double().cpu() <= 2 * bound).all()


@BOTH
def test_runs_repeat_bitwise(cuda_lib, splits):
    args = Case(2100, [5, 700, 0, 33], seed=70).args()
    assert torch.equal(decode(args, prefix_splits=splits)[0], decode(args, prefix_splits=splits)[0])


@BOTH
def test_bad_prefix_length_is_flagged_and_clamped(cuda_lib, splits):
    c = Case(64, [5, 33], seed=71)
    args = c.args()
    o, _ = decode(args, prefix_splits=splits)
    args[4].fill_(65)  # beyond the prefix's table
    got, st = decode(args, max_prefix_len=64, prefix_splits=splits)
    assert st == pda.DEV_BAD_SEQ_LEN and torch.equal(got, o)
    args[4].fill_(-2)
    got, st = decode(args, max_prefix_len=64, prefix_splits=splits)
    args[4].fill_(0)
    want, st0 = decode(args, max_prefix_len=64, prefix_splits=splits)
    assert st == pda.DEV_BAD_SEQ_LEN and st0 == 0 and torch.equal(got, want)


@BOTH
@pytest.mark.parametrize("page", [-1, 1 << 20])
def test_bad_prefix_page_is_flagged_and_reads_as_zeros(cuda_lib, page, splits):
    c = Case(200, [5, 33], seed=72)
    args = c.args()
    args[3][4] = page
    o, st = decode(args, prefix_splits=splits)
    assert st == pda.DEV_BAD_PAGE
    z = int(c.prefix_table[4])
    c.k[z] = 0
    c.v[z] = 0
    want, st = decode(c.args(), prefix_splits=splits)
    assert st == 0 and torch.equal(o, want)


@pytest.mark.parametrize("prefix_splits", [0, 1, 3])
def test_a_visible_nan_shows(cuda_lib, prefix_splits):
    c = Case(500, [5, 700], seed=73)
    clean, _ = decode(c.args(), prefix_splits=prefix_splits)
    page = int(c.prefix_table[7])
    keep = c.k[page].clone()
    c.k[page, 3] = float("nan")
    o, _ = decode(c.args(), prefix_splits=prefix_splits)
    assert torch.isnan(o).all()
    c.k[page] = keep
    c.k[int(c.table[1, 20]), 2] = float("nan")
    o, _ = decode(c.args(), prefix_splits=prefix_splits)
    assert torch.isnan(o[1]).all() and torch.equal(o[0], clean[0])


# (the bounds size the launches only: with the last ones every sequence has a block)
@pytest.mark.parametrize("kernels,max_prefix,max_seq,splits", [(3, 1008, 704, 2), (2, 1008, 704, 0), (1, 16, 16, 0)])
def test_streams_graphs_and_steps(cuda_lib, kernels, max_prefix, max_seq, splits):
    # two captured graphs and a step share one workspace in turn; lengths and contents change between replays
    args = Case(1000, [5, 700, 0, 33], seed=74).args()
    ws = pda.new_workspace(pda.attn_decode_prefix_workspace_size(4, max_prefix, max_seq, 0, splits), DEV)
    bounds = dict(max_prefix_len=max_prefix, max_seq_len=max_seq, prefix_splits=splits)
    kw = dict(bounds, workspace=ws, out_dtype=torch.float32)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(pda.attn_decode_global_prefix(*args, **kw))
        graphs.append(g)
    step = pda.Step()
    outs.append(step.add_decode_global_prefix(*args, **kw))
    assert step.num_kernels == kernels
    step.finalize("graph")
    call = pda.prepare_decode_global_prefix(*args, **kw)
    for prefix, lens in ((1000, [5, 700, 0, 33]), (17, [0, 16, 0, 20]), (640, [3, 600, 0, 33])):
        args[4].fill_(prefix)
        args[6].copy_(torch.tensor(lens, dtype=torch.int32))
        args[0].mul_(0.5)
        # (no length above goes beyond the first ones, whose pages are mapped)
        torch.cuda.synchronize()
        want, st = decode(args, **bounds)
        assert st == 0 and torch.isfinite(want).all()
        for g in graphs:
            g.replay()
        step.launch()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            got = call.run(side)
        torch.cuda.synchronize()
        for o in outs + [got]:
            assert torch.equal(o, want)
    step.close()


def test_serving_run_prefix_prompt_then_decode_steps(cuda_lib):
    # the prefix enters the cache once, a prompt of its own per sequence follows behind it, then decode steps
    g = torch.Generator().manual_seed(75)
    D, prefix, own, steps = 512, 83, [5, 0, 40], 2
    B, width = 3, 4
    pb = -(-prefix // 16)
    P = pb + B * width + 2
    perm = torch.randperm(P, generator=g).to(torch.int32)
    pt, bt = perm[:pb].to(DEV), perm[pb:pb + B * width].view(B, width).contiguous().to(DEV)
    k = torch.full((P, 16, 1, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    w_q, w_k = ((1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV) for _ in range(2))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    new = lambda n: torch.randn((n, append_row_len("global")), generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pda.attn_kv_append_global_chunk(new(prefix), w_q, w_k, pt[None], i32(prefix), i32(0, prefix), k, v, status=st)
    lens = i32(*own)
    pda.attn_kv_append_global_chunk(new(45), w_q, w_k, bt, lens, i32(0, 5, 5, 45), k, v, status=st)
    qkv, cu, plen = new(B), torch.arange(B + 1, dtype=torch.int32, device=DEV), i32(prefix)
    step = pda.Step()
    q = step.add_kv_append_global_chunk(qkv, w_q, w_k, bt, lens, cu, k, v, status=st)
    o = step.add_decode_global_prefix(q, k, v, pt, plen, bt, lens, out_dtype=torch.float32, status=st)
    step.finalize()
    for _ in range(steps):
        qkv.copy_(new(B))
        lens += 1
        step.launch()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        want, A, S = attention_rows(q, k, v, bt, lens, 0, prefix=(pt, prefix))
        bound = decode_bound(want, A, S, D, torch.float32, WEIGHT_EPS)
        assert ((o.double().cpu() - want).abs() <= bound).all()
    step.close()
