"""NaN and infinities that nodes see, in attn_decode_{sliding,global}_tree, on a GPU: several at once, in rows that every node
sees and in rows that some do, for whole and cut sequences, against IEEE arithmetic in 64 bits on what each node sees."""

import math

import pytest
import torch

import paged_decode_attention_gb300 as pda

from _fp8 import decode_bound
from _tree import TreeCase, chain, run_tree

pytestmark = pytest.mark.gpu

NAN, INF = math.nan, math.inf
KINDS = ["sliding", "global"]
#            0
#        1       2          6
#      3   4   5
TREE = [-1, 0, 0, 1, 1, 2, -1]
# context of the first sequence, num_splits: whole, and cut in few parts and many
CUTS = [(200, 0), (700, 0), (700, 16), (700, 60), (700, 152), (700, 1024)]


def ieee(c):
    """The outputs over what each node sees and nothing else [T, Hq, D], in 64 bits."""
    o = torch.empty((c.T, c.Hq, c.D), dtype=torch.float64)
    at = 0
    for b, n in enumerate(c.n):
        seen = c.seen(b)
        page, row = c.slot(b, torch.arange(c.lo[b], c.L[b]))
        k, v = c.k[page, row].double(), c.v[page, row].double()
        for i in range(n):
            for h in range(c.Hq):
                kv = h // (c.Hq // c.Hkv)
                w = torch.softmax(k[seen[i], kv] @ c.q[at + i, h].double(), 0)
                o[at + i, h] = (w[:, None] * v[seen[i], kv]).sum(0)
        at += n
    return o


def check(c, clean, out_dtype=torch.float32, **kw):
    """clean: want() of the case before its bad elements."""
    want = ieee(c)
    o, A, S = clean
    got, st = run_tree(pda, c, out_dtype, **kw)
    assert st == 0
    x = got[:c.T].double().cpu()
    finite = torch.isfinite(want)
    assert not finite.all()
    off = (x - o).abs() <= decode_bound(o, A, S, c.D, out_dtype, 2.0 ** -8)
    assert off[finite].all()
    assert torch.equal(x.isnan(), want.isnan())
    signed = want.isinf()
    assert torch.equal(x[signed], want[signed])


def test_the_cases_are_whole_and_cut():
    for kind in (pda.KIND_SLIDING, pda.KIND_GLOBAL):
        for ctx, splits in CUTS:
            launches = pda.attn_decode_tree_plan(kind, 2, 7, ctx + 7, 1024 if kind == pda.KIND_SLIDING else 0, splits)[1]
            assert launches == (1 if ctx == 200 else 2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("context,node", [(NAN, INF), (-INF, INF), (INF, INF), (INF, -INF), (INF, NAN), (-INF, -INF)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_values_that_all_and_that_some_nodes_see(cuda_lib, kind, context, node, out_dtype):
    for ctx, splits in CUTS:
        c = TreeCase(kind, [ctx, 40], [TREE, chain(3)], seed=41)
        clean = c.want()
        page, row = c.slot(0, torch.tensor([ctx - 50, ctx + 1, ctx + 5]))
        c.v[page[0], row[0], :, 33] = context
        c.v[page[1], row[1], :, 33] = node       # node 1 and those behind it
        c.v[page[2], row[2], :, 34] = node       # another dim, node 5
        c.v[page[0], row[0], :, c.D - 1] = context
        check(c, clean, out_dtype, num_splits=splits)


@pytest.mark.parametrize("kind", KINDS)
def test_a_key_that_all_nodes_see_and_a_value_that_some_do(cuda_lib, kind):
    for ctx, splits in CUTS:
        c = TreeCase(kind, [ctx, 40], [TREE, chain(3)], seed=42)
        clean = c.want()
        page, row = c.slot(0, torch.tensor([ctx - 50, ctx + 1]))
        c.k[page[0], row[0]] = NAN
        c.v[page[1], row[1], :, 33] = INF
        check(c, clean, num_splits=splits)


@pytest.mark.parametrize("kind", KINDS)
def test_two_values_of_one_path(cuda_lib, kind):
    """Infinities of both signs in rows that some nodes see: NaN for those behind both."""
    for ctx, splits in CUTS:
        c = TreeCase(kind, [ctx, 40], [TREE, chain(3)], seed=43)
        clean = c.want()
        page, row = c.slot(0, torch.tensor([ctx + 1, ctx + 4]))
        c.v[page[0], row[0], :, 5] = INF
        c.v[page[1], row[1], :, 5] = -INF
        check(c, clean, num_splits=splits)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("far", [100, 199])
def test_an_infinity_of_no_weight_does_not_depend_on_the_cut(cuda_lib, kind, out_dtype, far):
    """One key's scores stand some 250 above all others, so that every other weight is below fp32's range; `far` of a
    context of 200, or of 1200 for the cut cases.  The infinity stands in a node's row, behind the key."""
    for ctx, splits in CUTS:
        ctx = ctx if ctx == 200 else 1200
        c = TreeCase(kind, [ctx, 40], [TREE, chain(3)], seed=44)
        c.q[:, :, 0] = 1.0
        page, row = c.slot(0, torch.tensor([ctx - 200 + far, ctx + 1]))
        c.k[page[0], row[0], :, 0] = 256.0
        clean = c.want()
        c.v[page[1], row[1], :, 33] = INF
        check(c, clean, out_dtype, num_splits=splits)


@pytest.mark.parametrize("ahead", [100, 900, 1022])
def test_an_infinity_at_the_window_s_edge_does_not_depend_on_the_cut(cuda_lib, ahead):
    """The same for the first position that nodes of depth 0 see, in front of the key by `ahead`."""
    for splits in (0, 16, 60, 152, 1024):
        c = TreeCase("sliding", [1500, 40], [[-1, 0, -1, 1], chain(3)], seed=45)
        c.q[:, :, 0] = 1.0
        page, row = c.slot(0, torch.tensor([1500 - 1023, 1500 - 1023 + ahead]))
        c.k[page[1], row[1], :, 0] = 256.0
        clean = c.want()
        c.v[page[0], row[0], :, 33] = -INF
        check(c, clean, num_splits=splits)
