"""attn_decode_{sliding,global}_tree against the definition in 64 bits, on a GPU.

The bound is _fp8.decode_bound's for weights rounded to bf16 (2^-8 relative).  Every pool row that no node sees holds NaN,
so anything read from there shows."""

import pytest
import torch

import paged_decode_attention_gb300 as pda
from workloads import PAGE_SIZE

from _fp8 import decode_bound
from _tree import DEV, TreeCase, chain, random_tree, rng, run_tree, star

pytestmark = pytest.mark.gpu

WEIGHT = 2.0 ** -8


def check(c, out_dtype=torch.float32, **kw):
    got, st = run_tree(pda, c, out_dtype, **kw)
    assert st == 0
    o, A, S = c.want()
    x = got[:c.T].double().cpu()
    assert torch.isfinite(x).all()
    bound = decode_bound(o, A, S, c.D, out_dtype, WEIGHT)
    bad = (x - o).abs() > bound
    assert not bad.any(), "%d of %d off, worst %.3g of the bound" % (bad.sum(), bad.numel(),
                                                                    ((x - o).abs() / bound).max())
    assert (got[c.T:] == 7.0).all()
    return got


KINDS = ["sliding", "global"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ctx,n", [(0, 1), (1, 1), (15, 1), (16, 2), (127, 1), (128, 5), (200, 17), (700, 33), (900, 64)])
def test_one_sequence(cuda_lib, kind, ctx, n):
    check(TreeCase(kind, [ctx], [random_tree(n, rng(n + ctx))], seed=ctx + n))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_ragged_batch(cuda_lib, kind, out_dtype):
    r = rng(5)
    ctx = [0, 5, 3000, 16, 1023, 1024, 1025, 77, 400, 2048]
    trees = [random_tree(n, r) for n in (1, 64, 7, 0, 12, 16, 33, 4, 5, 2)]
    check(TreeCase(kind, ctx, trees, seed=11, spare=5), out_dtype)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [chain, star])
@pytest.mark.parametrize("n", [3, 16, 17, 64])
def test_chains_and_stars(cuda_lib, kind, shape, n):
    check(TreeCase(kind, [100, 1500], [shape(n), shape(max(1, n - 1))], seed=n))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 2, 5, 16, 100, 128, 1000])
def test_windows(cuda_lib, kind, window):
    """Windows inside a tree's depth, at page and step borders."""
    r = rng(window)
    trees = [chain(40), random_tree(64, r), star(9), random_tree(20, r), chain(1)]
    check(TreeCase(kind, [130, 900, 0, window, max(0, window - 1)], trees, seed=window, window=window))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits", [16, 17, 40, 152, 400, 1024])
def test_any_split_gives_the_same(cuda_lib, kind, splits):
    r = rng(splits)
    c = TreeCase(kind, [6000 if kind == "global" else 1100, 129, 0, 2222], [random_tree(n, r) for n in (9, 64, 3, 18)],
                 seed=21)
    check(c, num_splits=splits)


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences(cuda_lib, kind):
    r = rng(3)
    ctx = [r.randint(0, 300) for _ in range(256)]
    trees = [random_tree(r.choice([0, 1, 2, 3, 5, 8]), r) for _ in range(256)]
    check(TreeCase(kind, ctx, trees, seed=33), torch.bfloat16)


@pytest.mark.parametrize("kind", KINDS)
def test_large_logits_move_the_reference(cuda_lib, kind):
    """Scores of a standard deviation of 40 and more: references move, sums span many powers of two."""
    c = TreeCase(kind, [3000, 800], [random_tree(9, rng(1)), chain(20)], seed=8, scale=16.0)
    check(c, num_splits=16)
    rising = TreeCase(kind, [1000], [chain(5)], seed=9, scale=4.0)  # keys that grow along the context
    page, row = rising.slot(0, torch.arange(rising.lo[0], rising.L[0]))
    rising.k[page, row] = (rising.k[page, row].float() * torch.linspace(0.1, 12, page.shape[0])[:, None, None]).to(
        torch.bfloat16)
    check(rising, num_splits=16)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["k", "v"])
def test_what_a_node_does_not_see_is_not_used(cuda_lib, kind, bad, where):
    """A bad element in one node's row reaches that node and those behind it, and no others."""
    #            0
    #        1       2
    #      3   4   5
    parents = [-1, 0, 0, 1, 1, 2, -1]
    below = {2: {2, 5}, 4: {4}, 0: {0, 1, 2, 3, 4, 5}, 6: {6}}
    for node, hit in below.items():
        c = TreeCase(kind, [250, 40], [parents, chain(3)], seed=node)
        o, A, S = c.want()
        page, row = c.slot(0, torch.tensor([250 + node]))
        (c.k if where == "k" else c.v)[page, row, :, 17] = bad
        got, st = run_tree(pda, c, num_splits=16)
        assert st == 0
        x = got.double().cpu()
        clean = [i for i in range(c.T) if i not in hit]
        assert ((x - o).abs() <= decode_bound(o, A, S, c.D, torch.float32, WEIGHT))[clean].all()
        dirty = x[sorted(hit)]
        if where == "v":
            assert torch.isfinite(dirty[..., 16]).all() and torch.isfinite(dirty[..., 18:]).all()
            assert (dirty[..., 17].isnan() if bad != bad else dirty[..., 17] == bad).all()
        elif bad != bad:
            assert dirty.isnan().all()
        else:  # a score of an infinity's sign: no weight at all, or nothing but NaN
            assert (dirty.isnan().all(-1) | torch.isfinite(dirty).all(-1)).all()


def test_the_window_edge_is_not_used_by_deeper_nodes(cuda_lib):
    """The context's first visible position is seen by nodes of depth 0 only."""
    c = TreeCase("sliding", [1500], [[-1, 0, -1, 1]], seed=4)
    o, A, S = c.want()
    page, row = c.slot(0, torch.tensor([1500 - 1023]))
    c.v[page, row, :, 5] = float("nan")
    got, st = run_tree(pda, c)
    assert st == 0
    x = got.double().cpu()
    assert x[[0, 2]][..., 5].isnan().all()
    ok = (x - o).abs() <= decode_bound(o, A, S, c.D, torch.float32, WEIGHT)
    assert ok[[1, 3]].all()


@pytest.mark.parametrize("kind", KINDS)
def test_a_visible_nan_shows_in_cut_and_whole_sequences(cuda_lib, kind):
    for splits in (0, 16, 152):
        c = TreeCase(kind, [1000, 600], [chain(4), chain(2)], seed=6)
        page, row = c.slot(0, torch.tensor([700]))
        c.k[page, row] = float("nan")
        x = run_tree(pda, c, num_splits=splits)[0].cpu()
        assert x[:4].isnan().all() and torch.isfinite(x[4:]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_bad_pages_and_lengths_are_reported(cuda_lib, kind):
    trees = [chain(3), chain(2), chain(4)]
    c = TreeCase(kind, [40, 20, 30], trees, seed=12, fill=0.0)
    good = run_tree(pda, c)[0]
    for bad in (-1, c.P, 2 ** 30):
        keep = c.table.clone()
        c.table[1, 1] = bad
        got, st = run_tree(pda, c)
        assert st == pda.DEV_BAD_PAGE
        assert torch.equal(got[:3], good[:3]) and torch.equal(got[5:], good[5:]) and torch.isfinite(got).all()
        c.table = keep
    for b, length in ((1, 1), (1, -5), (1, 10 ** 6), (0, 2)):
        keep = c.lens.clone()
        c.lens[b] = length
        got, st = run_tree(pda, c)
        c.lens = keep
        assert st == pda.DEV_BAD_SEQ_LEN
        rows = slice(0, 3) if b == 0 else slice(3, 5)
        assert (got[rows] == 7.0).all()
        others = [i for i in range(9) if not rows.start <= i < rows.stop]
        assert torch.equal(got[others], good[others])
    got, st = run_tree(pda, c, max_q=3)  # more nodes than the host said
    assert st == pda.DEV_BAD_SEQ_LEN and (got[5:] == 7.0).all() and torch.equal(got[:5], good[:5])
    keep = c.cu.clone()
    c.cu[2] = 2  # decreases
    got, st = run_tree(pda, c)
    c.cu = keep
    assert st == pda.DEV_BAD_SEQ_LEN and (got == 7.0).all()
    c.cu[3] = 10  # past total_q
    got, st = run_tree(pda, c)
    assert st == pda.DEV_BAD_SEQ_LEN and (got[5:] == 7.0).all() and torch.equal(got[:5], good[:5])


@pytest.mark.parametrize("kind", KINDS)
def test_parents_outside_their_range_count_as_roots(cuda_lib, kind):
    want = run_tree(pda, TreeCase(kind, [50], [[-1, -1, 0, -1]], seed=2))[0]
    for bad in (-2, 1, 3, 2 ** 31 - 1, -2 ** 31):
        c = TreeCase(kind, [50], [[-1, -1, 0, -1]], seed=2)
        c.parents[1] = bad
        got, st = run_tree(pda, c)
        assert st == pda.DEV_BAD_TREE and torch.equal(got, want)


@pytest.mark.parametrize("kind", KINDS)
def test_a_chain_is_the_multi_query_attention(cuda_lib, kind):
    c = TreeCase(kind, [500, 1300], [chain(64), chain(17)], seed=14, fill=0.0)
    q, k, v, table, lens, cu, _ = c.args()
    ref = getattr(pda, "attn_prefill_%s" % kind)(q, k, v, table, lens, cu, out_dtype=torch.float32)
    got, st = run_tree(pda, c)
    assert st == 0
    _, A, S = c.want()
    bound = decode_bound(ref.double().cpu(), A, S, c.D, torch.float32, WEIGHT)
    assert ((got - ref).double().cpu().abs() <= 2 * bound).all()


@pytest.mark.parametrize("kind", KINDS)
def test_prepared_captured_and_repeated_calls_agree(cuda_lib, kind):
    r = rng(9)
    c = TreeCase(kind, [900, 60, 2000], [random_tree(n, r) for n in (8, 20, 5)], seed=15)
    want, st = run_tree(pda, c)
    assert st == 0
    again, st = run_tree(pda, c, prepared=True)
    assert st == 0 and torch.equal(again, want)
    kw = dict(window=c.window, max_q=c.max_n, max_seq_len=max(c.L), out_dtype=torch.float32)
    call = getattr(pda, "prepare_decode_%s_tree" % kind)(*c.args(), **kw)
    call.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run()
    call.out.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(call.out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = c.args()
    torch.cuda.synchronize()
    got = getattr(pda, "attn_decode_%s_tree" % kind)(*args, stream=side, **kw)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", KINDS)
def test_no_nodes(cuda_lib, kind):
    c = TreeCase(kind, [40, 3], [[], []], seed=1, spare=4)
    c.max_n = 5
    got, st = run_tree(pda, c)
    assert st == 0 and (got == 7.0).all()
    c.q, c.parents = c.q[:0], c.parents[:0]
    got, st = run_tree(pda, c)
    assert st == 0 and got.shape[0] == 0
    assert pda.attn_decode_tree_plan(pda.KIND_GLOBAL, 1, 0, 0, 0)[0] >= 1


@pytest.mark.parametrize("kind", KINDS)
def test_bounds_only_size_the_launch(cuda_lib, kind):
    """Defaults for max_q and max_seq_len, and bounds that are too small for the lengths."""
    c = TreeCase(kind, [1500, 20], [chain(5), star(6)], seed=31)
    want = check(c)
    got, st = run_tree(pda, c, max_q=None, max_seq_len=None)
    assert st == 0
    _, A, S = c.want()
    bound = decode_bound(want.double().cpu(), A, S, c.D, torch.float32, WEIGHT)
    assert ((got - want).double().cpu().abs() <= 2 * bound).all()
    assert PAGE_SIZE == 16


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("max_seq_len", [0, 1, 16, 200])
def test_many_sequences_longer_than_the_bound(cuda_lib, kind, max_seq_len):
    """More sequences than blocks, of more pages than the bound has: cut as any others."""
    r = rng(max_seq_len)
    n = 40 if kind == "sliding" else 200
    trees = [random_tree(r.choice([1, 2, 3, 4]), r) for _ in range(n)]
    check(TreeCase(kind, [r.randint(0, 600) for _ in range(n)], trees, seed=max_seq_len), max_seq_len=max_seq_len)
