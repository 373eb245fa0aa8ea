"""attn_decode_{sliding,global}_tree told of no nodes (max_q or total_q 0): lengths that deny it are reported, on a GPU."""

import pytest
import torch

import paged_decode_attention_gb300 as pda

from _tree import DEV, TreeCase, chain, run_tree

pytestmark = pytest.mark.gpu

KINDS = ["sliding", "global"]


def bad_cases(kind):
    """(case, max_q) whose lengths do not fit together."""
    yield TreeCase(kind, [40, 3], [chain(3), []], seed=1), 0              # nodes, and max_q 0
    yield TreeCase(kind, [0] * 255 + [9], [[]] * 255 + [chain(1)], seed=1), 0
    c = TreeCase(kind, [40, 3], [chain(3), []], seed=1)
    c.q, c.parents = c.q[:0], c.parents[:0]                               # rows past total_q
    yield c, 5
    c = TreeCase(kind, [40, 3], [[], []], seed=1, spare=2)
    c.lens[1] = c.table.shape[1] * 16 + 1                                 # beyond the table
    yield c, 0
    c = TreeCase(kind, [40, 3], [[], []], seed=1, spare=2)
    c.cu = torch.tensor([0, 2, 0], dtype=torch.int32)                     # decreases
    yield c, 0


@pytest.mark.parametrize("kind", KINDS)
def test_lengths_are_checked_without_nodes(cuda_lib, kind):
    for c, max_q in bad_cases(kind):
        got, st = run_tree(pda, c, max_q=max_q, max_seq_len=c.table.shape[1] * 16)
        assert st == pda.DEV_BAD_SEQ_LEN and (got == 7.0).all()
        got, st = run_tree(pda, c, max_q=max_q, max_seq_len=c.table.shape[1] * 16, status=None)
        assert (got == 7.0).all()
    c = TreeCase(kind, [40, 3, 0], [[], [], []], seed=1, spare=2)
    for max_q in (0, 4):
        got, st = run_tree(pda, c, max_q=max_q)
        assert st == 0 and (got == 7.0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("mode", ["direct", "graph"])
def test_in_a_step(cuda_lib, kind, mode):
    c = TreeCase(kind, [40, 3], [chain(3), []], seed=1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = c.args()
    for st, kernels in ((None, 0), (status, 1)):
        step = pda.Step()
        getattr(step, "add_decode_%s_tree" % kind)(*args, max_q=0, window=c.window, status=st)
        assert step.num_kernels == kernels
        step.finalize(mode)
        step.launch()
        torch.cuda.synchronize()
        assert int(status.item()) == (pda.DEV_BAD_SEQ_LEN if kernels else 0)
        step.close()
