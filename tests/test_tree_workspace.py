"""One workspace for a server's calls: attn_decode_tree_workspace_size of the largest covers every smaller one."""

import pytest
import torch

import paged_decode_attention_gb300 as pda

from _tree import DEV, TreeCase, random_tree, rng, run_tree

pytestmark = pytest.mark.gpu

KINDS = ["sliding", "global"]


def kind_of(kind):
    return pda.KIND_SLIDING if kind == "sliding" else pda.KIND_GLOBAL


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [0, 100, 1024])
@pytest.mark.parametrize("splits", [0, 16, 40])
def test_the_size_covers_smaller_arguments(cuda_lib, kind, window, splits):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    batches, nodes, lengths = (1, 2, 4, 8, 16, 19, 40, 256), (0, 1, 4, 5, 8, 9, 16, 17, 32, 33, 64), (0, 16, 100, 320, 600, 1100, 9000, 262144)
    window = window or (262144 if kind == "sliding" else 0)
    size = {(b, q, n): pda.attn_decode_tree_workspace_size(kind_of(kind), b, q, n, window, splits)
            for b in batches for q in nodes for n in lengths}
    for (b, q, n), s in size.items():
        needed = pda.attn_decode_tree_plan(kind_of(kind), b, q, n, window, splits, sms)[2]
        assert s >= needed
        for i, x in enumerate((b, q, n)):
            smaller = [y for y in (batches, nodes, lengths)[i] if y < x]
            if smaller:  # one step down in each argument; all others follow from these
                at = [b, q, n]
                at[i] = smaller[-1]
                assert size[tuple(at)] <= s, (at, (b, q, n))


@pytest.mark.parametrize("kind", KINDS)
def test_a_server_s_workspace_serves_its_smaller_batches(cuda_lib, kind):
    window = 1024 if kind == "sliding" else 0
    need = pda.attn_decode_tree_workspace_size(kind_of(kind), 16, 9, 320, window)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    for batch in (16, 8, 4, 1):
        for n in (9, 8, 4, 1):
            r = rng(batch + n)
            c = TreeCase(kind, [305] + [r.randint(0, 300) for _ in range(batch - 1)], [random_tree(n, r) for _ in range(batch)], seed=n)
            for max_seq_len in (320, max(c.L)):
                got, st = run_tree(pda, c, workspace=ws, max_seq_len=max_seq_len)
                want, _ = run_tree(pda, c, max_seq_len=max_seq_len)
                assert st == 0 and torch.equal(got, want)
