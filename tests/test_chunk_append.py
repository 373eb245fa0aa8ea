"""Chunk appends (attn_kv_append_*_chunk) and their 8-bit form (attn_kv_append_*_fp8) against the definition in 64 bits.

bf16 results are held to half a bf16 step plus the fp32 error of _fp8.ROW_EPS;
8-bit results to half an e4m3 step, or half a step of its smallest values at
the row's scale, plus the same.  Everything the call does not own keeps its
bytes.
"""

import numpy as np
import pytest
import torch

import paged_decode_attention_gb300 as pda
from workloads import GLOBAL, PAGE_SIZE, SLIDING, append_row_len

from _fp8 import E8, F8, ROW_EPS, append_rows, dequantise, quantise

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SHAPE = {"sliding": SLIDING, "global": GLOBAL}


class Chunk:
    """new[b] tokens of a sequence of L[b]; `spare` rows behind the last sequence."""

    def __init__(self, kind, L, new, seed, spare=0, scale=1.0, extra_pages=3):
        sh = SHAPE[kind]
        self.kind, self.L, self.new = kind, L, new
        self.Hq, self.Hkv, self.D = sh["Hq"], sh["Hkv"], sh["D"]
        g = torch.Generator().manual_seed(seed)
        T = sum(new)
        self.T = T
        self.qkv = (scale * torch.randn((T + spare, append_row_len(kind)), generator=g)).to(torch.bfloat16)
        self.w_q = (1 + 0.1 * torch.randn(self.D, generator=g)).to(torch.bfloat16)
        self.w_k = (1 + 0.1 * torch.randn(self.D, generator=g)).to(torch.bfloat16)
        width = max(1, max((-(-x // PAGE_SIZE) for x in L), default=1))
        need = [(b, p) for b, (x, n) in enumerate(zip(L, new)) if n for p in range((x - n) // PAGE_SIZE,
                                                                                  -(-x // PAGE_SIZE))]
        self.P = len(need) + extra_pages
        perm = torch.randperm(self.P, generator=g).to(torch.int32)
        self.table = torch.full((len(L), width), -1, dtype=torch.int32)
        for i, (b, p) in enumerate(need):
            self.table[b, p] = perm[i]
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.cu = torch.from_numpy(cu)
        self.pos = np.concatenate([np.arange(x - n, x) for x, n in zip(L, new)] + [np.zeros(0, int)]).astype(int)
        seq = np.repeat(np.arange(len(L)), new)
        self.page = self.table.numpy()[seq, self.pos // PAGE_SIZE] if T else np.zeros(0, int)
        self.row = self.pos % PAGE_SIZE

    def common(self):
        t = lambda x: x.to(DEV)  # noqa: E731
        return [t(self.qkv), t(self.w_q), t(self.w_k), t(self.table),
                torch.tensor(self.L, dtype=torch.int32, device=DEV), t(self.cu)]

    def want(self):
        return append_rows(self.kind, self.qkv[:self.T], self.w_q, self.w_k, self.pos, self.Hq, self.Hkv, self.D)

    def bf16_pools(self):
        shape = (self.P, PAGE_SIZE, self.Hkv, self.D)
        return [torch.full(shape, v, dtype=torch.bfloat16, device=DEV) for v in (3.0, -5.0)]

    def fp8_cache(self):
        k, v, ks, vs = pda.new_fp8_cache(0 if self.kind == "sliding" else 1, self.P, DEV)
        for x, byte in ((k, 0x11), (v, 0x92), (ks, 120), (vs, 131)):
            x.view(torch.uint8).fill_(byte)
        return k, v, ks, vs

    def others(self):
        """Mask [P, 16] of the rows that the call does not own."""
        m = np.ones((self.P, PAGE_SIZE), bool)
        m[self.page, self.row] = False
        return m


def close(got, want, eps, what):
    got = np.asarray(got, dtype=np.float64)
    assert np.isfinite(got).all(), what
    bound = eps * np.abs(want) + ROW_EPS * np.abs(want).max(-1, keepdims=True) + 1e-38
    bad = np.abs(got - want) > bound
    assert not bad.any(), "%s: %d elements off; worst %.3g" % (what, bad.sum(), (np.abs(got - want) / bound).max())


def run_chunk(c, values_only=False, **kw):
    k, v = c.bf16_pools()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.full((c.qkv.shape[0], c.Hq, c.D), 7.0, dtype=torch.bfloat16, device=DEV)
    fn = getattr(pda, "attn_kv_append_%s_chunk" % c.kind)
    q = fn(*c.common(), None if values_only else k, v, q_out, status=st, **kw)
    assert q is q_out
    torch.cuda.synchronize()
    return q, k, v, int(st.item())


def check_chunk(c, **kw):
    q, k, v, st = run_chunk(c, **kw)
    assert st == 0
    wq, wk, wv = c.want()
    eps = torch.finfo(torch.bfloat16).eps / 2
    q, k, v = (x.double().cpu().numpy() for x in (q, k, v))
    close(q[:c.T], wq, eps, "q")
    assert (q[c.T:] == 7.0).all()
    close(k[c.page, c.row], wk, eps, "k")
    close(v[c.page, c.row], wv, eps, "v")
    m = c.others()
    assert (k[m] == 3.0).all() and (v[m] == -5.0).all()


def run_fp8(c, **kw):
    cache = c.fp8_cache()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.full((c.qkv.shape[0], c.Hq, c.D), 7.0, dtype=torch.bfloat16, device=DEV)
    fn = getattr(pda, "attn_kv_append_%s_fp8" % c.kind)
    fn(*c.common(), *cache, q_out, status=st, **kw)
    torch.cuda.synchronize()
    return q_out, cache, int(st.item())


def check_fp8(c):
    q, (k, v, ks, vs), st = run_fp8(c)
    assert st == 0
    wq, wk, wv = c.want()
    close(q.double().cpu().numpy()[:c.T], wq, torch.finfo(torch.bfloat16).eps / 2, "q")
    m = c.others()
    for codes, scales, want, other, other_scale in ((k, ks, wk, 0x11, 120), (v, vs, wv, 0x92, 131)):
        got = dequantise(codes, scales).cpu().numpy()[c.page, c.row]
        cb, sb = codes.view(torch.uint8).cpu().numpy(), scales.view(torch.uint8).cpu().numpy().transpose(0, 2, 1)
        s = sb[c.page, c.row].astype(np.int64) - 127
        want_codes, want_s = quantise(want)
        amax = np.abs(want).max(-1)
        # the scale: the smallest power of two that fits, but for rows within the fp32 error of a border
        border = np.abs(amax / (448.0 * 2.0 ** s) - 1) < ROW_EPS
        border |= np.abs(amax / (224.0 * 2.0 ** s) - 1) < ROW_EPS
        assert (border | (s + 127 == want_s)).all()
        bound = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * 2.0 ** s[..., None] + ROW_EPS * amax[..., None]
        assert (np.abs(got - want) <= bound).all()
        same = (cb[c.page, c.row] == want_codes)[~border]
        if same.size > 5000:
            # a code differs only where the value lies within the fp32 error (at most ROW_EPS of the row's largest, a
            # few steps' width of 2^-4 relative values) of a rounding border
            assert same.mean() > 0.999
        assert (cb[m] == other).all() and (sb[m] == other_scale).all()


CASES = [
    ("one token", [1], [1], 0),
    ("first of a page", [17], [1], 0),
    ("far position", [262144], [3], 0),
    ("whole prompt", [50], [50], 0),
    ("ragged", [1, 40, 16, 33, 300, 64, 5], [1, 7, 16, 17, 129, 0, 5], 4),
    ("empty sequences", [0, 9, 0, 0, 20, 0], [0, 2, 0, 0, 20, 0], 1),
]


@pytest.mark.parametrize("kind", ["sliding", "global"])
@pytest.mark.parametrize("label,L,new,spare", CASES, ids=[c[0] for c in CASES])
def test_chunk_matches_the_definition(cuda_lib, kind, label, L, new, spare):
    check_chunk(Chunk(kind, L, new, 11, spare))


@pytest.mark.parametrize("kind", ["sliding", "global"])
@pytest.mark.parametrize("label,L,new,spare", CASES, ids=[c[0] for c in CASES])
def test_fp8_matches_the_definition(cuda_lib, kind, label, L, new, spare):
    check_fp8(Chunk(kind, L, new, 12, spare))


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_full_batch_and_more_tokens_than_blocks(cuda_lib, kind):
    # 256 sequences with 0 to 7 tokens each, and 1500 tokens in one sequence: blocks take several tokens
    r = np.random.RandomState(3)
    new = r.randint(0, 8, 256).tolist()
    L = [n + int(r.randint(0, 90)) for n in new]
    check_chunk(Chunk(kind, L, new, 13))
    check_fp8(Chunk(kind, L, new, 14))
    check_chunk(Chunk(kind, [1700], [1500], 15))


@pytest.mark.parametrize("kind", ["sliding", "global"])
@pytest.mark.parametrize("scale", [2.0 ** -40, 1e-3, 2.0 ** 40])
def test_input_scales(cuda_lib, kind, scale):
    check_chunk(Chunk(kind, [40, 7], [9, 7], 16, scale=scale))
    check_fp8(Chunk(kind, [40, 7], [9, 7], 17, scale=scale))


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_one_token_each_equals_the_single_token_call(cuda_lib, kind):
    L = [1, 16, 17, 500, 4096]
    c = Chunk(kind, L, [1] * 5, 18)
    q, k, v, _ = run_chunk(c)
    k1, v1 = c.bf16_pools()
    a = c.common()
    positions = a[4] - 1
    q1 = getattr(pda, "attn_kv_append_%s" % kind)(a[0], a[1], a[2], a[3], positions, k1, v1)
    torch.cuda.synchronize()
    # The same fp32 steps but for their order and the products that form a pair's frequency: the fp32 values differ by
    # at most twice _fp8.ROW_EPS of the row's largest, and two values either side of a rounding border end one bf16
    # step apart, which is eps = 2^-7 of a value just above a power of two (not the 2^-8 of a rounding to nearest).
    for x, y in ((q, q1), (k, k1), (v, v1)):
        d = (x.double() - y.double()).abs()
        y = y.double().abs()
        assert (d <= torch.finfo(torch.bfloat16).eps * y + 2 * ROW_EPS * y.amax(-1, keepdim=True)).all()
        assert (d == 0).double().mean() > 0.999


def test_values_only_global_cache(cuda_lib):
    c = Chunk("global", [30, 5], [12, 5], 19)
    q, k, v, st = run_chunk(c, values_only=True)
    q2, _, v2, _ = run_chunk(c)
    assert st == 0 and torch.equal(q, q2) and torch.equal(v, v2) and (k == 3.0).all()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_a_row_with_nan_or_infinity_reads_as_nan(cuda_lib, kind):
    c = Chunk(kind, [4], [4], 20)
    off = c.Hq * c.D
    c.qkv[1, off + 3] = float("nan")
    c.qkv[2, off + 5] = float("inf")
    _, (k, v, ks, vs), st = run_fp8(c)
    assert st == 0
    kd = dequantise(k, ks).cpu().numpy()[c.page, c.row]
    vd = dequantise(v, vs).cpu().numpy()[c.page, c.row]
    for t, bad in ((0, False), (1, True), (2, True), (3, False)):
        assert np.isnan(kd[t, 0]).all() == bad and np.isnan(kd[t, 0]).any() == bad
        if kind == "global":  # one source row for both
            assert np.isnan(vd[t, 0]).all() == bad
        else:
            assert np.isfinite(kd[t, 1:]).all() and np.isfinite(vd[t]).all()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_a_row_of_zeros(cuda_lib, kind):
    c = Chunk(kind, [3], [3], 21)
    c.qkv[1] = 0
    q, (k, v, ks, vs), st = run_fp8(c)
    assert st == 0 and (q[1] == 0).all()
    for codes, scales in ((k, ks), (v, vs)):
        assert (codes.view(torch.uint8)[c.page[1], c.row[1]] & 127 == 0).all()
        assert (scales.view(torch.uint8)[c.page[1], :, c.row[1]] == 1).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_bad_lengths_and_pages_leave_their_rows_alone(cuda_lib, kind, fp8):
    def go(c):
        if fp8:
            q, (k, v, ks, vs), st = run_fp8(c)
            return q, k.view(torch.uint8), v.view(torch.uint8), st, 0x11
        q, k, v, st = run_chunk(c)
        return q, k, v, st, 3.0

    # more new tokens than the sequence holds: nothing of it is written, the others are
    c = Chunk(kind, [20, 20, 20], [5, 5, 5], 22)
    ok = go(c)
    c.L = [20, 4, 20]
    q, k, v, st, other = go(c)
    assert st == pda.DEV_BAD_SEQ_LEN
    assert (q[5:10] == 7.0).all() and torch.equal(q[:5], ok[0][:5]) and torch.equal(q[10:], ok[0][10:])
    assert (k[c.page[5:10], c.row[5:10]] == other).all()
    assert torch.equal(k[c.page[10:], c.row[10:]], ok[1][c.page[10:], c.row[10:]])
    # a length beyond the table
    c.L = [20, 33, 20]
    assert go(c)[3] == pda.DEV_BAD_SEQ_LEN
    # cu_q past the packed rows, and decreasing
    c.L = [20, 20, 20]
    c.cu = torch.tensor([0, 5, 10, 99], dtype=torch.int32)
    q, _, _, st, _ = go(c)
    assert st == pda.DEV_BAD_SEQ_LEN and (q[10:] == 7.0).all() and torch.equal(q[:10], ok[0][:10])
    c.cu = torch.tensor([0, 5, 3, 15], dtype=torch.int32)
    assert go(c)[3] & pda.DEV_BAD_SEQ_LEN
    # a bad page: the token's q is written, its cache row is not
    c.cu = torch.tensor([0, 5, 10, 15], dtype=torch.int32)
    c.table[1, 0] = c.P
    c.table[2, 0] = -1
    q, k, v, st, other = go(c)
    assert st == pda.DEV_BAD_PAGE and torch.equal(q, ok[0])
    first = np.nonzero(c.pos[10:] < PAGE_SIZE)[0] + 10
    assert (k[c.page[first], c.row[first]] == other).all() and (v[c.page[first], c.row[first]] == (0x92 if fp8 else
                                                                                                   -5.0)).all()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_no_tokens(cuda_lib, kind):
    c = Chunk(kind, [5, 0], [0, 0], 23)
    q, k, v, st = run_chunk(c)
    assert st == 0 and q.shape[0] == 0 and (k == 3.0).all()
    _, (k, _, _, _), st = run_fp8(c)
    assert st == 0 and (k.view(torch.uint8) == 0x11).all()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_captured_stream_and_step_replays_follow_their_inputs(cuda_lib, kind):
    c = Chunk(kind, [40, 3, 90], [8, 3, 1], 24)
    args = c.common()
    k, v = c.bf16_pools()
    cache = c.fp8_cache()
    q1 = torch.zeros((c.T, c.Hq, c.D), dtype=torch.bfloat16, device=DEV)
    q2 = torch.zeros_like(q1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        getattr(pda, "attn_kv_append_%s_chunk" % kind)(*args, k, v, q1)
    step = pda.Step()
    getattr(step, "add_kv_append_%s_fp8" % kind)(*args, *cache, q2)
    getattr(step, "add_kv_append_%s_chunk" % kind)(*args, k, v, q1)
    step.finalize("graph")
    for seed in (25, 26):
        other = Chunk(kind, [40, 3, 90], [8, 3, 1], seed)
        args[0].copy_(other.qkv)
        graph.replay()
        step.launch()
        torch.cuda.synchronize()
        c.qkv = other.qkv
        wq, wk, _ = c.want()
        close(q1.double().cpu().numpy(), wq, 2.0 ** -8, "captured")
        assert torch.equal(q1, q2)
        close(k.double().cpu().numpy()[c.page, c.row], wk, 2.0 ** -8, "captured k")
        got = dequantise(cache[0], cache[2]).cpu().numpy()[c.page, c.row]
        assert (np.abs(got - wk) <= 0.07 * np.abs(wk) + 2.0 ** -12 * np.abs(wk).max()).all()
    step.close()
