"""Refusals of the chunk appends, the 8-bit cache and the shared-prefix calls, without a GPU: error codes before anything is launched."""

import ctypes

import numpy as np
import pytest
import torch

import paged_decode_attention_gb300 as pda
from paged_decode_attention_gb300 import _build

from _fp8 import dequantise, e4m3_table, quantise

FAKE = 1 << 20  # an aligned, never dereferenced address
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pda.load()


ARGS = {
    "chunk": ["qkv", "w_q", "w_k", "table", "lens", "cu_q", "q_out", "k", "v", "batch", "total_q", "max_blocks",
              "num_pages", "status"],
    "fp8": ["qkv", "w_q", "w_k", "table", "lens", "cu_q", "q_out", "k", "v", "ks", "vs", "batch", "total_q",
            "max_blocks", "num_pages", "status"],
    "read": ["k", "v", "ks", "vs", "table", "lens", "k_out", "v_out", "out_table", "batch", "max_blocks", "num_pages",
             "out_pages", "max_seq_len", "span", "status"],
    "decode": ["q", "k", "v", "ks", "vs", "table", "lens", "o", "batch", "max_blocks", "num_pages", "max_seq_len",
               "window", "out_dtype", "num_splits", "ws", "ws_bytes", "status"],
    "prefix": ["q", "k", "v", "prefix_table", "prefix_len", "table", "lens", "o", "batch", "prefix_blocks",
               "max_blocks", "num_pages", "max_prefix_len", "max_seq_len", "out_dtype", "num_splits", "prefix_splits",
               "ws", "ws_bytes", "status"],
}
DEFAULTS = dict(batch=4, total_q=9, max_blocks=70, num_pages=300, out_pages=200, max_seq_len=1100, span=0, window=1024,
                out_dtype=0, num_splits=0, prefix_blocks=30, max_prefix_len=480, prefix_splits=0, ws=None, ws_bytes=0, status=None)
NAMES = {"attn_kv_append_%s_chunk": "chunk", "attn_kv_append_%s_fp8": "fp8", "attn_kv_read_%s_fp8": "read",
         "attn_decode_%s_fp8": "decode", "attn_decode_%s_prefix": "prefix"}


def call(lib, name, form, step=None, **kw):
    values = [kw.get(a, DEFAULTS.get(a, FAKE)) for a in ARGS[form]]
    if step is not None:
        return getattr(lib, name.replace("attn_", "attn_step_add_"))(step, *values)
    return getattr(lib, name)(*values, None)


def bad_calls():
    for pattern, form in NAMES.items():
        for kind in ("sliding", "global"):
            if form == "prefix" and kind == "sliding":
                continue
            name = pattern % kind
            pointers = [a for a in ARGS[form] if a not in DEFAULTS]
            for a in pointers:
                if not (a == "k" and form == "chunk" and kind == "global"):
                    yield name, form, {a: None}, INVALID
                yield name, form, {a: FAKE + 2}, INVALID
            yield name, form, dict(status=FAKE + 1), INVALID
            yield name, form, dict(batch=0), INVALID
            yield name, form, dict(batch=257), UNSUPPORTED
            yield name, form, dict(max_blocks=0), INVALID
            yield name, form, dict(num_pages=0), INVALID
            yield name, form, dict(num_pages=1 << 27), INVALID
            if form in ("chunk", "fp8"):
                yield name, form, dict(total_q=-1), INVALID
                yield name, form, dict(total_q=(1 << 28) + 1), UNSUPPORTED
            if form == "read":
                yield name, form, dict(out_pages=0), INVALID
            if form == "prefix":
                yield name, form, dict(prefix_blocks=0), INVALID
                yield name, form, dict(max_prefix_len=-1), INVALID
                yield name, form, dict(max_prefix_len=481), INVALID
                yield name, form, dict(prefix_blocks=20000, max_prefix_len=262145), UNSUPPORTED
                yield name, form, dict(prefix_splits=-1), INVALID
            if form in ("read", "decode", "prefix"):
                yield name, form, dict(max_seq_len=-1), INVALID
                yield name, form, dict(max_seq_len=70 * 16 + 1), INVALID
                yield name, form, dict(max_blocks=20000, max_seq_len=262145), UNSUPPORTED
            if form in ("decode", "prefix"):
                yield name, form, dict(out_dtype=2), INVALID
                yield name, form, dict(num_splits=-1), INVALID
                if kind == "sliding" and form == "decode":
                    yield name, form, dict(window=0), INVALID


@pytest.mark.parametrize("name,form,bad,code", list(bad_calls()), ids=lambda x: str(x))
def test_bad_arguments_are_refused_before_launch(lib, name, form, bad, code):
    assert call(lib, name, form, **bad) == code
    assert name in pda.attn_last_error()
    h = ctypes.c_void_p()
    assert lib.attn_step_create(ctypes.byref(h)) == 0
    try:
        assert call(lib, name, form, step=h, **bad) == code
        assert lib.attn_step_num_calls(h) == 0
    finally:
        lib.attn_step_destroy(h)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_no_tokens_is_a_call_without_a_launch(lib, kind):
    for suffix, form in (("chunk", "chunk"), ("fp8", "fp8")):
        assert call(lib, "attn_kv_append_%s_%s" % (kind, suffix), form, total_q=0, qkv=None, q_out=None) == 0


def test_fp8_plan(lib):
    S, G = pda.KIND_SLIDING, pda.KIND_GLOBAL

    def a256(x):
        return (x + 255) // 256 * 256

    # a block for every short sequence: a page and a virtual page each, two-page spans
    for kind, D, n in ((S, 256, 30), (G, 512, 30)):
        gx, _, ws = pda.attn_decode_fp8_plan(kind, n, 15, 1024 if kind == S else 0)
        assert gx == n
        rows = (gx + n) * 16
        assert ws == pda.WORKSPACE_ZERO_BYTES + a256(rows * D * 4) + a256(rows * 8)
    # one wave of resident blocks; long sequences keep four-page spans (250 pages + 1 -> 63 blocks)
    assert pda.attn_decode_fp8_plan(G, 4, 262144, 0)[0] == 304
    assert pda.attn_decode_fp8_plan(S, 256, 32768, 1024)[:2] == (57, 1)
    assert pda.attn_decode_fp8_plan(G, 1, 4000, 0)[:2] == (63, 2)
    assert pda.attn_decode_fp8_plan(G, 1, 0, 0)[0] == 1
    assert pda.attn_decode_fp8_plan(G, 2, 100, 0, num_splits=7)[0] == 7
    assert pda.attn_decode_fp8_plan(G, 2, 100, 0, num_splits=5000)[0] == 1024
    # short sequences whole, a block each, no merge
    for kind, n, longest in ((G, 1, 64), (G, 4, 128), (G, 64, 256), (G, 256, 512), (S, 57, 128)):
        window = 1024 if kind == S else 0
        assert pda.attn_decode_fp8_plan(kind, n, longest, window)[:2] == (n, 1)
        assert pda.attn_decode_fp8_plan(kind, n, longest, window, num_splits=7)[0] == 7
    assert pda.attn_decode_fp8_plan(G, 1, 65, 0)[:2] == (3, 2)
    assert pda.attn_decode_fp8_plan(G, 256, 513, 0)[:2] == (304, 2)
    assert pda.attn_decode_fp8_plan(S, 58, 16, 1024)[0] == 57
    for bad in ((7, 1, 16, 0), (G, 0, 16, 0), (G, 1, -1, 0), (G, 1, 16, 0, -1), (G, 1, 16, 0, 0, 0)):
        with pytest.raises(pda.AttnDecodeError):
            pda.attn_decode_fp8_plan(*bad)


def test_prefix_plan(lib):
    # 64 sequences: 4 pairs of query tiles x 2 slices = 8 clusters, 76 SM pairs -> 9 spans
    ns, ps, ws = pda.attn_decode_prefix_plan(64, 32768, 2048)
    own, _, own_ws = pda.attn_decode_fp8_plan(pda.KIND_GLOBAL, 64, 2048, 0)
    rows = ps * 64 * 16
    assert (ns, ps) == (own, 9) and ws == own_ws + rows * 512 * 4 + rows * 2 * 8
    # short prefixes, small batches: one list of pages per sequence, no spans
    for B, n in ((16, 1887), (8, 8450), (1, 262144), (2, 131072), (43, 2), (16, 0)):
        gx, ps, ws = pda.attn_decode_prefix_plan(B, n, 100)
        assert (gx, ps, ws) == (pda.attn_decode_fp8_plan(pda.KIND_GLOBAL, B, -(-n // 16) * 16 + 100, 0)[0], 0,
                                pda.attn_decode_fp8_plan(pda.KIND_GLOBAL, B, -(-n // 16) * 16 + 100, 0)[2])
    assert pda.attn_decode_prefix_plan(16, 1888, 100)[1] == 15  # spans of no less than two steps of 64 keys
    assert pda.attn_decode_prefix_plan(65, 0, 16)[1] == 1 and pda.attn_decode_prefix_plan(2, 2**31 - 1, 2**31 - 1)[1] == 0
    assert pda.attn_decode_prefix_plan(256, 262144, 16)[1] == 2
    assert pda.attn_decode_prefix_plan(8, 262144, 16, prefix_splits=7)[1] == 7
    assert pda.attn_decode_prefix_plan(8, 100, 16, prefix_splits=1)[1] == 1
    assert pda.attn_decode_prefix_plan(8, 262144, 16, prefix_splits=5000)[1] == 128
    for bad in ((0, 16, 16), (1, -1, 16), (1, 16, -1), (1, 16, 16, -1), (1, 16, 16, 0, -1), (1, 16, 16, 0, 0, 0)):
        with pytest.raises(pda.AttnDecodeError):
            pda.attn_decode_prefix_plan(*bad)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_binding_refuses_cpu_tensors(lib, kind):
    k = getattr(pda, "KIND_" + kind.upper())
    cache = pda.new_fp8_cache(k, 2, "cpu")
    Hq, Hkv, D = pda.SHAPES[k]
    assert cache[0].shape == (2, 16, Hkv, D) and cache[2].shape == (2, Hkv, 16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        getattr(pda, "attn_decode_%s_fp8" % kind)(bf(1, Hq, D), *cache, i32(1, 1), i32(1))
    with pytest.raises(ValueError, match="CUDA"):
        getattr(pda, "attn_kv_append_%s_fp8" % kind)(bf(1, pda.APPEND_ROW[k]), bf(D), bf(D), i32(1, 1), i32(1), i32(2),
                                                     *cache)
    pools = [bf(2, 16, Hkv, D), bf(2, 16, Hkv, D)]
    with pytest.raises(ValueError, match="CUDA"):
        getattr(pda, "attn_kv_append_%s_chunk" % kind)(bf(1, pda.APPEND_ROW[k]), bf(D), bf(D), i32(1, 1), i32(1),
                                                       i32(2), *pools)
    with pytest.raises(ValueError, match="CUDA"):
        getattr(pda, "attn_kv_read_%s_fp8" % kind)(*cache, i32(1, 1), i32(1), *pools)
    if kind == "global":
        with pytest.raises(ValueError, match="CUDA"):
            pda.attn_decode_global_prefix(bf(1, Hq, D), *pools, i32(1), i32(1), i32(1, 1), i32(1))
    step = pda.Step()
    with pytest.raises(ValueError, match="CUDA"):
        getattr(step, "add_decode_%s_fp8" % kind)(bf(1, Hq, D), *cache, i32(1, 1), i32(1))
    assert step.num_calls == 0
    step.close()


def test_the_plain_format_agrees_with_torch():
    # e4m3 as torch reads it, and the quantiser's rounding on torch's conversion of the scaled values
    codes = torch.arange(256, dtype=torch.uint8)
    assert torch.allclose(codes.view(torch.float8_e4m3fn).double(), e4m3_table(), equal_nan=True, rtol=0, atol=0)
    r = np.random.RandomState(1)
    y = r.standard_normal((400, 64)) * np.exp(r.uniform(-20, 20, (400, 1)))
    y[3] = 0
    y[4, 2] = np.nan
    y[5, :] = 448.0 * 2.0 ** 3
    y[6, :] = np.nextafter(448.0, 500)
    c, s = quantise(y)
    k = s.astype(np.int64) - 127
    assert s[3] == 1 and s[4] == 255 and k[5] == 3 and k[6] == 1
    ok = np.arange(400) != 4
    z = torch.from_numpy(y[ok] / 2.0 ** k[ok, None])
    assert np.array_equal(z.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy(), c[ok])
    back = dequantise(torch.from_numpy(c.reshape(25, 16, 1, 64)), torch.from_numpy(s.reshape(25, 1, 16)))
    err = np.abs(back.numpy().reshape(400, 64) - y)[ok]
    assert (err <= 2.0 ** -4 * np.abs(y[ok]) + 2.0 ** -10 * 2.0 ** k[ok, None]).all()
