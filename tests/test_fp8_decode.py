"""Decode over an 8-bit cache (attn_decode_*_fp8) and its read-back (attn_kv_read_*_fp8) against the definition in 64
bits over the dequantised cache, element by element within _fp8.decode_bound.  Every slot that a query may not read is
NaN (code 0x7f, scale 255)."""

import numpy as np
import pytest
import torch

import paged_decode_attention_gb300 as pda
from workloads import GLOBAL, PAGE_SIZE, SLIDING, append_row_len, make_case

from _fp8 import E8, F8, Fp8Case, attention_rows, decode_bound, dequantise

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
KINDS = ["sliding", "global"]
WEIGHT_EPS = torch.finfo(torch.float16).eps / 2


def decode(kind, args, window, status=None, **kw):
    st = torch.zeros(1, dtype=torch.int32, device=DEV) if status is None else status
    kw.setdefault("out_dtype", torch.float32)
    o = getattr(pda, "attn_decode_%s_fp8" % kind)(*args, window=window, status=st, **kw)
    torch.cuda.synchronize()
    return o, int(st.item())


def reference(args, window):
    q, k, v, ks, vs, bt, sl = args
    return attention_rows(q, dequantise(k, ks), dequantise(v, vs), bt, sl, window, v_scale=vs)


def check(kind, args, window, label="", **kw):
    o, st = decode(kind, args, window, **kw)
    assert st == 0, "%s: status %d" % (label, st)
    want, A, S, Q, F = reference(args, window)
    bound = decode_bound(want, A, S, args[0].shape[2], o.dtype, WEIGHT_EPS, Q, F)
    got = o.double().cpu()
    assert torch.isfinite(got).all(), label
    err = (got - want).abs()
    assert (err <= bound).all(), "%s: %.3g times the bound" % (label, float((err / bound).max()))
    return o


def window_of(kind):
    return 1024 if kind == "sliding" else 0


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", KINDS)
def test_edge_lengths(cuda_lib, kind, out_dtype):
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 48, 49, 64, 65, 1023, 1024, 1025, 1039, 1040, 1041]
    c = Fp8Case(make_case(kind, lens, seed=31))
    o = check(kind, c.on(DEV), window_of(kind), out_dtype=out_dtype)
    assert (o[0] == 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_one_position_returns_its_value(cuda_lib, kind):
    c = Fp8Case(make_case(kind, [1, 17], seed=32, window=1))
    args = c.on(DEV)
    o, st = decode(kind, args, 1)
    assert st == 0
    v = dequantise(args[2], args[4]).cpu()
    for b, pos in ((0, 0), (1, 16)):
        row = v[int(c.block_table[b, pos // 16]), pos % 16].repeat_interleave(16 // v.shape[2], 0)
        # the one weight is 1; in f16 and times the scale it is exact, so the value comes back exactly
        assert torch.equal(o[b].double().cpu(), row)


@pytest.mark.parametrize("window", [1, 7, 16, 17, 100, 1000])
@pytest.mark.parametrize("kind", KINDS)
def test_windows(cuda_lib, kind, window):
    c = Fp8Case(make_case(kind, [1, 40, 999, 2100], seed=33, window=window, window_only=True))
    check(kind, c.on(DEV), window)


@pytest.mark.parametrize("num_splits", [1, 3, 64, 1000])
@pytest.mark.parametrize("kind", KINDS)
def test_forced_splits(cuda_lib, kind, num_splits):
    c = Fp8Case(make_case(kind, [3, 700, 1100, 2500, 0], seed=34))
    check(kind, c.on(DEV), window_of(kind), num_splits=num_splits)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens", [[1], [64], [0, 0, 33], [16, 17, 0, 128, 1, 100], [5] * 57])
@pytest.mark.parametrize("kind", KINDS)
def test_short_sequences_whole(cuda_lib, kind, lens, out_dtype):
    c = Fp8Case(make_case(kind, lens, seed=50, window=window_of(kind)))
    assert pda.attn_decode_fp8_plan(pda.KIND_GLOBAL if kind == "global" else pda.KIND_SLIDING, len(lens), max(lens),
                                    window_of(kind))[:2] == (len(lens), 1)
    for bound in (max(lens), 1):  # (the bound sizes the launch only)
        o = check(kind, c.on(DEV), window_of(kind), out_dtype=out_dtype, max_seq_len=bound)
        for b, n in enumerate(lens):
            assert n or (o[b] == 0).all()


def test_a_large_batch_whole(cuda_lib):
    lens = torch.randint(0, 300, (200,), generator=torch.Generator().manual_seed(51)).tolist()
    c = Fp8Case(make_case("global", lens, seed=51, window=0))
    check("global", c.on(DEV), 0, max_seq_len=300)


@pytest.mark.parametrize("lens", [[20000], [0, 17000], [1, 6001], [9000, 0, 5]])
@pytest.mark.parametrize("num_splits", [0, 500])
def test_long_sequences_in_many_partials(cuda_lib, lens, num_splits):
    c = Fp8Case(make_case("global", lens, seed=49, window=0))
    check("global", c.on(DEV), 0, num_splits=num_splits)


@pytest.mark.parametrize("kind", KINDS)
def test_full_batch_of_mixed_lengths(cuda_lib, kind):
    r = np.random.RandomState(35)
    lens = [int(x) for x in np.exp(r.uniform(0, np.log(400), 256))]
    lens[7] = lens[100] = 0
    check(kind, Fp8Case(make_case(kind, lens, seed=35)).on(DEV), window_of(kind))


@pytest.mark.parametrize("kind", KINDS)
def test_scales_that_differ_from_row_to_row(cuda_lib, kind):
    # value scales of 2^-30 .. 2^30, growing and falling along the sequence, and key scales over 2^-6 .. 2^1
    c = Fp8Case(make_case(kind, [700, 45, 2000], seed=36, window=0 if kind == "global" else 1024))
    g = torch.Generator().manual_seed(36)
    live_v, live_k = c.vs != 255, c.ks != 255
    c.vs = torch.where(live_v, torch.randint(97, 158, c.vs.shape, generator=g).to(torch.uint8), c.vs)
    c.ks = torch.where(live_k, torch.randint(116, 123, c.ks.shape, generator=g).to(torch.uint8), c.ks)
    check(kind, c.on(DEV), window_of(kind))
    # the smallest and the largest scales (values near both ends of fp32's range): 1, 254
    for byte in (1, 120, 235):
        c.vs = torch.where(live_v, torch.full_like(c.vs, byte), c.vs)
        check(kind, c.on(DEV), window_of(kind), label="scale %d" % byte)


@pytest.mark.parametrize("exponent", [-60, -20, 15, 60])
@pytest.mark.parametrize("kind", KINDS)
def test_query_range_beyond_f16(cuda_lib, kind, exponent):
    # q times 2^e and the keys' scales times 2^-e leave the logits as they were
    c = Fp8Case(make_case(kind, [300, 17, 1500], seed=37))
    base = c.on(DEV)
    o, _ = decode(kind, base, window_of(kind))
    args = list(base)
    args[0] = (base[0].double() * 2.0 ** exponent).to(torch.bfloat16)
    ks = base[3].view(torch.uint8)
    args[3] = torch.where(ks == 255, ks, (ks.int() - exponent).to(torch.uint8)).view(E8)
    got, st = decode(kind, args, window_of(kind))
    assert st == 0 and torch.equal(got, o)


@pytest.mark.parametrize("kind", KINDS)
def test_flat_and_dominated_weights(cuda_lib, kind):
    c = Fp8Case(make_case(kind, [1500, 33], seed=38))
    args = c.on(DEV)
    zero = [torch.zeros_like(args[0])] + list(args[1:])
    check(kind, zero, window_of(kind), label="flat")
    big = [(args[0].float() * 20).to(torch.bfloat16)] + list(args[1:])
    check(kind, big, window_of(kind), label="dominated")


@pytest.mark.parametrize("num_splits", [0, 1, 40])
@pytest.mark.parametrize("kind", KINDS)
def test_a_visible_nan_shows_and_stays_in_its_sequence(cuda_lib, kind, num_splits):
    c = Fp8Case(make_case(kind, [500, 500, 700], seed=39))
    clean, _ = decode(kind, c.on(DEV), window_of(kind), num_splits=num_splits)
    page, row = int(c.block_table[1, 20]), 3
    for what in ("k scale", "v scale", "k code", "v code"):
        c2 = Fp8Case(c.base)
        if what == "k scale":
            c2.ks[page, 0, row] = 255
        elif what == "v scale":
            c2.vs[page, 0, row] = 255
        elif what == "k code":
            c2.k[page, row, 0, 9] = 0x7f
        else:
            c2.v[page, row, 0, 9] = 0xff
        o, st = decode(kind, c2.on(DEV), window_of(kind), num_splits=num_splits)
        G = 16 // c2.k.shape[2]
        hit = o[1, :G]
        assert torch.isnan(hit[..., 9] if what == "v code" else hit).all(), what
        o[1, :G] = clean[1, :G]
        assert torch.equal(o, clean), what


@pytest.mark.parametrize("kind", KINDS)
def test_paging_is_a_relabelling_and_runs_repeat_bitwise(cuda_lib, kind):
    c = Fp8Case(make_case(kind, [3, 16, 17, 700, 1500], seed=40))
    oa, _ = decode(kind, c.on(DEV), window_of(kind))
    ob, _ = decode(kind, c.on(DEV), window_of(kind))
    assert torch.equal(oa, ob)
    perm = torch.randperm(c.k.shape[0], generator=torch.Generator().manual_seed(9))
    for name in ("k", "v", "ks", "vs"):
        x = getattr(c, name)
        y = torch.empty_like(x)
        y[perm] = x
        setattr(c, name, y)
    args = list(c.on(DEV))
    bt = c.block_table.clone()
    m = bt >= 0
    bt[m] = perm[bt[m].long()].to(torch.int32)
    args[5] = bt.to(DEV)
    oc, _ = decode(kind, args, window_of(kind))
    assert torch.equal(oa, oc)


@pytest.mark.parametrize("kind", KINDS)
def test_bad_page_is_flagged_and_reads_as_zeros(cuda_lib, kind):
    c = Fp8Case(make_case(kind, [100, 40], seed=41))
    args = list(c.on(DEV))
    P = c.k.shape[0]
    page0, page1 = int(c.block_table[0, 2]), int(c.block_table[1, 0])
    bt = args[5].clone()
    bt[0, 2], bt[1, 0] = -1, P + 5
    o, st = decode(kind, args[:5] + [bt, args[6]], window_of(kind))
    assert st == pda.DEV_BAD_PAGE
    for x in (c.k, c.v):
        x[page0] = 0
        x[page1] = 0
    for x in (c.ks, c.vs):
        x[page0] = 0
        x[page1] = 0
    z, st = decode(kind, c.on(DEV), window_of(kind))
    assert st == 0 and torch.equal(o, z)


@pytest.mark.parametrize("kind", KINDS)
def test_bad_length_is_flagged(cuda_lib, kind):
    c = Fp8Case(make_case(kind, [100, 40], seed=42))
    args = list(c.on(DEV))
    args[6] = torch.tensor([-3, 40], dtype=torch.int32, device=DEV)
    o, st = decode(kind, args, window_of(kind), max_seq_len=100)
    assert st == pda.DEV_BAD_SEQ_LEN and (o[0] == 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_pages_beyond_32_bit_offsets(cuda_lib, kind):
    # a pool of more than 2^31 bytes, whose last pages hold the sequence
    sh = SLIDING if kind == "sliding" else GLOBAL
    page_bytes = PAGE_SIZE * sh["Hkv"] * sh["D"]
    small = Fp8Case(make_case(kind, [60], seed=43))
    n = small.k.shape[0]
    P = (1 << 31) // page_bytes + 3 + n
    args = list(small.on(DEV))
    big = []
    for x in args[1:5]:
        y = torch.zeros((P,) + tuple(x.shape[1:]), dtype=torch.uint8, device=DEV)
        y[P - n:] = x.view(torch.uint8)
        big.append(y.view(x.dtype))
    bt = torch.where(args[5] >= 0, args[5] + (P - n), args[5])
    want, _ = decode(kind, args, window_of(kind))
    got, st = decode(kind, [args[0]] + big + [bt, args[6]], window_of(kind))
    assert st == 0 and torch.equal(got, want)
    out = [torch.zeros((n, PAGE_SIZE, sh["Hkv"], sh["D"]), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    getattr(pda, "attn_kv_read_%s_fp8" % kind)(*big, bt, args[6], *out, args[5])
    torch.cuda.synchronize()
    pos = torch.arange(60)
    page = small.block_table[0, pos // 16].long()
    assert torch.equal(out[0].double().cpu()[page, pos % 16],
                       dequantise(args[1], args[3]).cpu()[page, pos % 16])


@pytest.mark.parametrize("span", [0, 1, 16, 100, 5000])
@pytest.mark.parametrize("kind", KINDS)
def test_read_back_is_exact_and_touches_nothing_else(cuda_lib, kind, span):
    lens = [0, 1, 16, 17, 100, 333, 1200]
    c = Fp8Case(make_case(kind, lens, seed=44, window=span if span else 0, window_only=span > 0))
    args = c.on(DEV)
    P, width = c.k.shape[0], c.block_table.shape[1]
    g = torch.Generator().manual_seed(44)
    # other pages out than in
    out_pages = P + 5
    perm = torch.randperm(out_pages, generator=g).to(torch.int32)
    table = torch.where(c.block_table >= 0, perm[c.block_table.clamp(min=0).long()], c.block_table)
    shape = (out_pages,) + tuple(c.k.shape[1:])
    k_out, v_out = (torch.full(shape, x, dtype=torch.bfloat16, device=DEV) for x in (3.0, -5.0))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ret = getattr(pda, "attn_kv_read_%s_fp8" % kind)(*args[1:], k_out, v_out, table.to(DEV), span=span, status=st)
    assert ret[0] is k_out and ret[1] is v_out
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    want_k, want_v = torch.full(shape, 3.0, dtype=torch.float64), torch.full(shape, -5.0, dtype=torch.float64)
    kd, vd = dequantise(args[1], args[3]).cpu(), dequantise(args[2], args[4]).cpu()
    for b, L in enumerate(lens):
        pos = torch.arange(max(0, L - span) if span > 0 else 0, L)
        src, dst = c.block_table[b, pos // 16].long(), table[b, pos // 16].long()
        want_k[dst, pos % 16] = kd[src, pos % 16]
        want_v[dst, pos % 16] = vd[src, pos % 16]
    assert torch.equal(k_out.double().cpu(), want_k) and torch.equal(v_out.double().cpu(), want_v)
    assert width == table.shape[1]


def test_read_back_flags_bad_pages(cuda_lib):
    c = Fp8Case(make_case("global", [40, 20], seed=45))
    args = list(c.on(DEV))
    out = [torch.full(tuple(c.k.shape), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for where in ("in", "out"):
        bad = args[5].clone()
        bad[0, 1] = -1 if where == "in" else c.k.shape[0]
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        tables = (bad, args[6]) if where == "in" else (args[5], args[6])
        pda.attn_kv_read_global_fp8(*args[1:5], *tables, *out, args[5] if where == "in" else bad, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == pda.DEV_BAD_PAGE
        page = int(c.block_table[0, 1])
        assert (out[0][page] == 3.0).all() and (out[0][int(c.block_table[1, 0])] != 3.0).any()


@pytest.mark.parametrize("kind", KINDS)
def test_read_back_prepared_and_in_a_step(cuda_lib, kind):
    c = Fp8Case(make_case(kind, [70, 5, 300], seed=48))
    args = list(c.on(DEV))
    shape = tuple(c.k.shape)
    outs = [[torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2)] for _ in range(3)]
    name = "kv_read_%s_fp8" % kind
    call = getattr(pda, "prepare_" + name)(*args[1:], *outs[1], span=100)
    step = pda.Step()
    getattr(step, "add_" + name)(*args[1:], *outs[2], span=100)
    step.finalize()
    for lens in ([70, 5, 300], [3, 0, 290]):  # contents change between runs
        args[6].copy_(torch.tensor(lens, dtype=torch.int32))
        getattr(pda, "attn_" + name)(*args[1:], *outs[0], span=100)
        assert call.run()[0] is outs[1][0]
        step.launch()
        torch.cuda.synchronize()
        for o in outs[1:]:
            assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])
    step.close()


@pytest.mark.parametrize("bound", [1300, 40])  # (sizes the launch only: 40 gives every sequence a block)
@pytest.mark.parametrize("kind", KINDS)
def test_streams_graphs_and_steps(cuda_lib, kind, bound):
    # the same workspace by two captured graphs and a step in turn, contents changing between replays
    lens = [5, 700, 1300, 64]
    cases = [Fp8Case(make_case(kind, lens, seed=46 + i, layout_seed=46)) for i in range(3)]
    args = list(cases[0].on(DEV))
    w = window_of(kind)
    ws = pda.new_workspace(pda.attn_decode_fp8_workspace_size(getattr(pda, "KIND_" + kind.upper()), 4, bound, w), DEV)
    kw = dict(window=w, max_seq_len=bound, workspace=ws, out_dtype=torch.float32)
    fn = getattr(pda, "attn_decode_%s_fp8" % kind)
    side = torch.cuda.Stream()
    graphs, outs = [], []
    torch.cuda.synchronize()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs.append(fn(*args, **kw))
        graphs.append(graph)
    step = pda.Step()
    outs.append(getattr(step, "add_decode_%s_fp8" % kind)(*args, **kw))
    step.finalize("graph")
    call = getattr(pda, "prepare_decode_%s_fp8" % kind)(*args, **kw)
    for c in cases:
        new = c.on(DEV)
        for x, y in zip(args, new):
            if x.element_size() == 1:
                x.view(torch.uint8).copy_(y.view(torch.uint8))
            else:
                x.copy_(y)
        torch.cuda.synchronize()
        want, _ = decode(kind, new, w, max_seq_len=bound)
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


@pytest.mark.parametrize("kind", KINDS)
def test_serving_run_prompt_read_back_prefill_and_decode_steps(cuda_lib, kind):
    # a prompt enters the 8-bit cache, is read back for the prefill's attention, and three decode steps follow, each an
    # append and a decode recorded as one step
    sh = SLIDING if kind == "sliding" else GLOBAL
    Hq, Hkv, D, w = sh["Hq"], sh["Hkv"], sh["D"], sh["window"]
    prompt, steps = [70, 1, 1100], 3
    B = len(prompt)
    g = torch.Generator().manual_seed(47)
    width = -(-(max(prompt) + steps) // 16)
    P = B * width + 1
    table = torch.randperm(P, generator=g)[:B * width].view(B, width).to(torch.int32).to(DEV)
    cache = pda.new_fp8_cache(getattr(pda, "KIND_" + kind.upper()), P, DEV)
    for x in cache[:2]:
        x.view(torch.uint8).fill_(0x7f)
    for x in cache[2:]:
        x.view(torch.uint8).fill_(255)
    w_q, w_k = ((1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV) for _ in range(2))
    row = append_row_len(kind)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(prompt)]), dtype=torch.int32, device=DEV)
    lens = torch.tensor(prompt, dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    qkv = torch.randn((sum(prompt), row), generator=g).to(torch.bfloat16).to(DEV)
    q = getattr(pda, "attn_kv_append_%s_fp8" % kind)(qkv, w_q, w_k, table, lens, cu, *cache, status=st)
    out = [torch.full((P, 16, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    getattr(pda, "attn_kv_read_%s_fp8" % kind)(*cache, table, lens, *out, status=st)
    o = getattr(pda, "attn_prefill_%s" % kind)(q, out[0], out[1], table, lens, cu, window=w, max_q=max(prompt),
                                               out_dtype=torch.float32, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    kd, vd = dequantise(cache[0], cache[2]), dequantise(cache[1], cache[3])
    for b, t, n in ((0, 69, 70), (1, 70, 1), (2, 71 + 1099, 1100), (2, 71 + 500, 501)):  # last queries, and a middle one
        want, A, S = attention_rows(q[t:t + 1], kd, vd, table[b:b + 1], [n], w)
        bound = decode_bound(want, A, S, D, torch.float32, torch.finfo(torch.bfloat16).eps / 2)
        assert ((o[t:t + 1].double().cpu() - want).abs() <= bound).all()
    # decode steps
    qkv1 = torch.zeros((B, row), dtype=torch.bfloat16, device=DEV)
    cu1 = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    step = pda.Step()
    q1 = getattr(step, "add_kv_append_%s_fp8" % kind)(qkv1, w_q, w_k, table, lens, cu1, *cache, status=st)
    o1 = getattr(step, "add_decode_%s_fp8" % kind)(q1, *cache, table, lens, window=w, out_dtype=torch.float32,
                                                  status=st)
    step.finalize()
    for i in range(steps):
        qkv1.copy_(torch.randn((B, row), generator=g).to(torch.bfloat16))
        lens += 1
        step.launch()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        want, A, S, Q, F = attention_rows(q1, dequantise(cache[0], cache[2]), dequantise(cache[1], cache[3]), table,
                                          lens, w, v_scale=cache[3])
        bound = decode_bound(want, A, S, D, torch.float32, WEIGHT_EPS, Q, F)
        assert ((o1.double().cpu() - want).abs() <= bound).all()
    step.close()
