"""Tokens behind a shared prefix: attn_kv_append_global_prefix (attn_kv_append_global_chunk with prefix_len) puts them
where attn_decode_global_prefix looks for them and rotates them where they stand, for prefixes of any length."""

import ctypes

import numpy as np
import pytest
import torch

import paged_decode_attention_gb300 as pda
from paged_decode_attention_gb300 import _build
from workloads import PAGE_SIZE, append_row_len

from _fp8 import append_rows, attention_rows, decode_bound
from test_chunk_append import Chunk, close, run_chunk

DEV = "cuda:0"
FAKE = 1 << 20  # an aligned, never dereferenced address
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2


# ---------------------------------------------------------------------------
# refusals, without a GPU
# ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pda.load()


ARGS = ["qkv", "w_q", "w_k", "prefix_len", "table", "lens", "cu_q", "q_out", "k", "v", "batch", "total_q", "max_blocks",
        "num_pages", "status"]
POINTERS = ARGS[:10]
GOOD = dict(dict.fromkeys(POINTERS, FAKE), batch=4, total_q=9, max_blocks=70, num_pages=300, status=None)
BAD = [({a: None}, 1) for a in POINTERS] + [({a: FAKE + 2}, 1) for a in POINTERS] + [
    (dict(status=FAKE + 1), 1), (dict(batch=0), 1), (dict(batch=257), 2), (dict(max_blocks=0), 1), (dict(num_pages=0), 1),
    (dict(num_pages=1 << 27), 1), (dict(total_q=-1), 1), (dict(total_q=(1 << 28) + 1), 2)]


@pytest.mark.parametrize("bad,code", BAD, ids=str)
def test_bad_arguments_are_refused_before_launch(lib, bad, code):
    values = [dict(GOOD, **bad)[a] for a in ARGS]
    assert lib.attn_kv_append_global_prefix(*values, None) == code
    assert "attn_kv_append_global_prefix" in pda.attn_last_error()
    h = ctypes.c_void_p()
    assert lib.attn_step_create(ctypes.byref(h)) == 0
    try:
        assert lib.attn_step_add_kv_append_global_prefix(h, *values) == code
        assert lib.attn_step_num_calls(h) == 0
    finally:
        lib.attn_step_destroy(h)


def test_the_binding_refuses_what_has_no_such_form(lib):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(TypeError):
        pda.attn_kv_append_sliding_chunk(*[i32(1)] * 8, prefix_len=i32(1))
    with pytest.raises(TypeError):
        pda.attn_kv_append_global_fp8(*[i32(1)] * 10, prefix_len=i32(1))


@pytest.mark.gpu
def test_the_binding_checks_prefix_len(cuda_lib):
    c = Chunk("global", [5], [5], 100)
    k, v = c.bf16_pools()
    for bad, error in ((torch.zeros(1, dtype=torch.int32), ValueError),
                       (torch.zeros(1, dtype=torch.int64, device=DEV), TypeError),
                       (torch.zeros(2, dtype=torch.int32, device=DEV), ValueError)):
        with pytest.raises(error):
            pda.attn_kv_append_global_chunk(*c.common(), k, v, prefix_len=bad)
    with pytest.raises(TypeError):  # a values-only cache rebuilds its keys at their positions in the table
        pda.attn_kv_append_global_chunk(*c.common(), None, v, prefix_len=torch.zeros(1, dtype=torch.int32, device=DEV))
    s = Chunk("sliding", [5], [5], 100)
    k, v = s.bf16_pools()
    with pytest.raises(ValueError, match="global"):
        pda.prepare_kv_append_sliding_chunk(*s.common(), k, v,
                                            prefix_len=torch.zeros(1, dtype=torch.int32, device=DEV))


# ---------------------------------------------------------------------------
# against the definition in 64 bits
# ---------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 5003, 262144])
def test_tokens_are_rotated_behind_the_prefix_and_cached_at_their_own_positions(cuda_lib, prefix):
    c = Chunk("global", [1, 40, 16, 33, 300, 0], [1, 7, 16, 17, 129, 0], 101, spare=3)
    n = torch.tensor([prefix], dtype=torch.int32, device=DEV)
    q, k, v, st = run_chunk(c, prefix_len=n)
    assert st == 0
    wq, wk, wv = append_rows("global", c.qkv[:c.T], c.w_q, c.w_k, c.pos + prefix, c.Hq, c.Hkv, c.D)
    q, k, v = (x.double().cpu().numpy() for x in (q, k, v))
    close(q[:c.T], wq, BF16_HALF, "q")
    assert (q[c.T:] == 7.0).all()
    close(k[c.page, c.row], wk, BF16_HALF, "k")
    close(v[c.page, c.row], wv, BF16_HALF, "v")
    m = c.others()
    assert (k[m] == 3.0).all() and (v[m] == -5.0).all()


@pytest.mark.gpu
def test_no_prefix_is_the_plain_append_and_bad_lengths_write_nothing(cuda_lib):
    c = Chunk("global", [20, 40], [5, 40], 102)
    plain = run_chunk(c)
    for n, ok in ((0, True), (-1, False), (262145, False)):
        got = run_chunk(c, prefix_len=torch.tensor([n], dtype=torch.int32, device=DEV))
        if ok:
            assert got[3] == 0 and all(torch.equal(x, y) for x, y in zip(got[:3], plain[:3]))
        else:
            assert got[3] == pda.DEV_BAD_SEQ_LEN and (got[0] == 7.0).all()
            assert (got[1] == 3.0).all() and (got[2] == -5.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("pages", [1, 7])
def test_behind_whole_pages_it_is_the_append_through_joined_tables(cuda_lib, pages):
    c = Chunk("global", [40, 90, 3], [8, 33, 3], 103)
    q, k, v, st = run_chunk(c, prefix_len=torch.tensor([16 * pages], dtype=torch.int32, device=DEV))
    assert st == 0
    # the same rows at absolute positions: the prefix's pages (never touched) in front of the own
    c.table = torch.cat([torch.full((3, pages), -1, dtype=torch.int32), c.table], 1).contiguous()
    c.L = [x + 16 * pages for x in c.L]
    q2, k2, v2, st = run_chunk(c)
    assert st == 0 and torch.equal(q, q2) and torch.equal(k, k2) and torch.equal(v, v2)


@pytest.mark.gpu
@pytest.mark.parametrize("prefix", [83, 96, 5003])
@pytest.mark.parametrize("splits", [0, 2])
def test_serving_run_behind_a_prefix_against_the_definition(cuda_lib, prefix, splits):
    # the prefix enters once, an own prompt per sequence behind it, then decode steps (append and decode, one step); every
    # cached key and every query is held to the definition at its place in the whole text
    g = torch.Generator().manual_seed(104)
    D, own, steps, width = 512, [5, 0, 40], 3, 4
    B, pb = len(own), -(-prefix // PAGE_SIZE)
    P = pb + B * width + 2
    perm = torch.randperm(P, generator=g).to(torch.int32)
    pt, bt = perm[:pb].to(DEV), perm[pb:pb + B * width].view(B, width).contiguous().to(DEV)
    k = torch.full((P, PAGE_SIZE, 1, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    w_q, w_k = ((1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV) for _ in range(2))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    new = lambda n: torch.randn((n, append_row_len("global")), generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    plen = i32(prefix)

    def hold(qkv, positions, q, pages, rows):
        wq, wk, wv = append_rows("global", qkv, w_q, w_k, positions, 16, 1, D)
        at = lambda pool: pool[torch.as_tensor(pages).long(), torch.as_tensor(rows)].double().cpu().numpy()  # noqa: E731
        close(q.double().cpu().numpy(), wq, BF16_HALF, "q")
        close(at(k.cpu()), wk, BF16_HALF, "k")
        close(at(v.cpu()), wv, BF16_HALF, "v")

    text = new(prefix)
    q = pda.attn_kv_append_global_chunk(text, w_q, w_k, pt[None], plen, i32(0, prefix), k, v, status=st)
    pos = np.arange(prefix)
    hold(text, pos, q, pt.cpu()[pos // 16], pos % 16)
    lens = i32(*own)
    prompt = new(45)
    q = pda.attn_kv_append_global_chunk(prompt, w_q, w_k, bt, lens, i32(0, 5, 5, 45), k, v, prefix_len=plen, status=st)
    seq, pos = np.repeat(np.arange(B), own), np.concatenate([np.arange(n) for n in own])
    hold(prompt, prefix + pos, q, bt.cpu()[seq, pos // 16], pos % 16)
    qkv, cu = new(B), torch.arange(B + 1, dtype=torch.int32, device=DEV)
    step = pda.Step()
    q = step.add_kv_append_global_chunk(qkv, w_q, w_k, bt, lens, cu, k, v, prefix_len=plen, status=st)
    o = step.add_decode_global_prefix(q, k, v, pt, plen, bt, lens, out_dtype=torch.float32, prefix_splits=splits,
                                      status=st)
    step.finalize()
    for _ in range(steps):
        qkv.copy_(new(B))
        lens += 1
        step.launch()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        pos = lens.cpu().numpy() - 1
        hold(qkv, prefix + pos, q, bt.cpu()[np.arange(B), pos // 16], pos % 16)
        want, A, S = attention_rows(q, k, v, bt, lens, 0, prefix=(pt, prefix))
        assert ((o.double().cpu() - want).abs() <= decode_bound(want, A, S, D, torch.float32, BF16_HALF)).all()
    step.close()


@pytest.mark.gpu
def test_prepared_captured_and_follows_the_length_on_the_device(cuda_lib):
    c = Chunk("global", [40, 3, 90], [8, 3, 1], 105)
    args, n = c.common(), torch.tensor([83], dtype=torch.int32, device=DEV)
    k, v = c.bf16_pools()
    q = torch.zeros((c.T, c.Hq, c.D), dtype=torch.bfloat16, device=DEV)
    call = pda.prepare_kv_append_global_chunk(*args, k, v, q, prefix_len=n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pda.attn_kv_append_global_chunk(*args, k, v, q, prefix_len=n)
    for prefix, go in ((83, call.run), (5003, graph.replay), (17, call.run), (16, graph.replay)):
        n.fill_(prefix)
        go()
        torch.cuda.synchronize()
        wq, wk, _ = append_rows("global", c.qkv, c.w_q, c.w_k, c.pos + prefix, c.Hq, c.Hkv, c.D)
        close(q.double().cpu().numpy(), wq, BF16_HALF, "q")
        close(k.double().cpu().numpy()[c.page, c.row], wk, BF16_HALF, "k")
