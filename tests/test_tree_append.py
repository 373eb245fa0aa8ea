"""attn_kv_append_{sliding,global}_tree: nodes cached at their slots, rotated at the context's length plus their depth."""

import numpy as np
import pytest
import torch

import paged_decode_attention_gb300 as pda

from _fp8 import append_rows
from _tree import DEV, chain, chains_of, random_tree, rng, star
from test_chunk_append import Chunk, close, run_chunk

pytestmark = pytest.mark.gpu

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2


def run_append(c, parents, **kw):
    k, v = c.bf16_pools()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.full((c.qkv.shape[0], c.Hq, c.D), 7.0, dtype=torch.bfloat16, device=DEV)
    p = torch.tensor(parents + [0] * (c.qkv.shape[0] - len(parents)), dtype=torch.int32, device=DEV)
    q = getattr(pda, "attn_kv_append_%s_tree" % c.kind)(*c.common(), p, k, v, q_out, status=st, **kw)
    assert q is q_out
    torch.cuda.synchronize()
    return q, k, v, int(st.item())


def turned(c, trees):
    """Position of every node in its text."""
    return np.concatenate([np.array([x - n + len(up) - 1 for up in chains_of(t)], dtype=int)
                           for x, n, t in zip(c.L, c.new, trees)] + [np.zeros(0, int)])


@pytest.mark.parametrize("kind", ["sliding", "global"])
@pytest.mark.parametrize("shape", ["random", "chain", "star", "roots"])
def test_nodes_are_rotated_at_their_depth(cuda_lib, kind, shape):
    new = [1, 64, 0, 33, 7, 2, 32]
    L = [1, 64, 9, 20000, 23, 17, 262144]
    make = {"random": lambda n: random_tree(n, rng(n)), "chain": chain, "star": star,
            "roots": lambda n: [-1] * n}[shape]
    trees = [make(n) for n in new]
    c = Chunk(kind, L, new, 61, spare=3)
    q, k, v, st = run_append(c, [p for t in trees for p in t])
    assert st == 0
    wq, wk, wv = append_rows(kind, c.qkv[:c.T], c.w_q, c.w_k, turned(c, trees), c.Hq, c.Hkv, c.D)
    q, k, v = (x.double().cpu().numpy() for x in (q, k, v))
    close(q[:c.T], wq, BF16_HALF, "q")
    assert (q[c.T:] == 7.0).all()
    close(k[c.page, c.row], wk, BF16_HALF, "k")
    close(v[c.page, c.row], wv, BF16_HALF, "v")
    m = c.others()
    assert (k[m] == 3.0).all() and (v[m] == -5.0).all()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_a_chain_is_the_chunk_append(cuda_lib, kind):
    new = [5, 64, 1]
    c = Chunk(kind, [40, 64, 3000], new, 62)
    a, b = run_append(c, [p for n in new for p in chain(n)]), run_chunk(c)
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3])) and a[3] == b[3] == 0


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_faults_are_reported(cuda_lib, kind):
    c = Chunk(kind, [40, 65, 30], [4, 65, 2], 63)  # more nodes than a tree may have
    good = chain(4), chain(65), chain(2)
    q, k, v, st = run_append(c, [p for t in good for p in t])
    assert st == pda.DEV_BAD_SEQ_LEN
    assert (q[4:69] == 7.0).all() and not (q[:4] == 7.0).all(-1).any() and not (q[69:] == 7.0).all(-1).any()
    c = Chunk(kind, [40, 30], [4, 3], 64)
    want = run_append(c, [-1, -1, 0, 2, -1, 0, 0])
    for bad in (1, 2, -2, 2 ** 31 - 1, -2 ** 31):
        got = run_append(c, [-1, bad, 0, 2, -1, 0, 0])
        assert got[3] == pda.DEV_BAD_TREE and all(torch.equal(x, y) for x, y in zip(got[:3], want[:3]))
    c.table[1, 1] = c.P
    got = run_append(c, [-1, -1, 0, 2, -1, 0, 0])
    assert got[3] == pda.DEV_BAD_PAGE and torch.equal(got[0], want[0])
