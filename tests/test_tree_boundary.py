"""Refusals of the tree calls, the commit and the page assignment, and the tree plan, without a GPU."""

import ctypes
import os
import subprocess

import pytest
import torch

import paged_decode_attention_gb300 as pda
from paged_decode_attention_gb300 import _build

FAKE = 1 << 20  # an aligned, never dereferenced address
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pda.load()


class Pools(list):
    """A host array of pool pointers."""


ARGS = {
    "tree": ["q", "k", "v", "table", "lens", "cu_q", "parents", "o", "batch", "total_q", "max_q", "max_blocks",
             "num_pages", "max_seq_len", "window", "out_dtype", "num_splits", "ws", "ws_bytes", "status"],
    "append": ["qkv", "w_q", "w_k", "table", "lens", "cu_q", "parents", "q_out", "k", "v", "batch", "total_q",
               "max_blocks", "num_pages", "status"],
    "commit": ["ks", "vs", "layers", "table", "lens", "cu_q", "path", "path_len", "new_lens", "batch", "max_path",
               "max_blocks", "num_pages", "status"],
    "assign": ["cached", "new", "table", "held", "free_list", "free_state", "held_out", "free_state_out", "seq_lens",
               "cu_q", "batch", "max_blocks", "num_pages", "window", "status"],
}
DEFAULTS = dict(batch=4, total_q=9, max_q=5, max_blocks=70, num_pages=300, max_seq_len=1100, window=1024, out_dtype=0,
                num_splits=0, ws=FAKE, ws_bytes=1 << 40, status=None, layers=2, max_path=8,
                ks=Pools([FAKE, 2 * FAKE]), vs=Pools([3 * FAKE, 4 * FAKE]))
NAMES = {"attn_decode_%s_tree": "tree", "attn_kv_append_%s_tree": "append", "attn_kv_commit_%s": "commit"}


def call(lib, name, form, step=None, **kw):
    values = [kw.get(a, DEFAULTS.get(a, FAKE)) for a in ARGS[form]]
    keep = [(ctypes.c_void_p * len(v))(*v) if isinstance(v, Pools) else v for v in values]
    values = [ctypes.cast(v, ctypes.c_void_p) if isinstance(v, ctypes.Array) else v for v in keep]
    if step is not None:
        return getattr(lib, name.replace("attn_", "attn_step_add_"))(step, *values)
    return getattr(lib, name)(*values, None)


def bad_calls():
    names = [(p % k, f, k) for p, f in NAMES.items() for k in ("sliding", "global")] + [("attn_pages_assign", "assign", "")]
    for name, form, kind in names:
        for a in ARGS[form]:
            if a not in DEFAULTS or a in ("ks", "vs"):
                yield name, form, {a: None}, INVALID
                yield name, form, {a: FAKE + 2}, INVALID
        if form == "assign":
            for a in ("held", "free_state", "held_out", "free_state_out"):
                yield name, form, {a: FAKE + 4}, INVALID
        yield name, form, dict(status=FAKE + 1), INVALID
        yield name, form, dict(batch=0), INVALID
        yield name, form, dict(batch=257), UNSUPPORTED
        yield name, form, dict(max_blocks=0), INVALID
        yield name, form, dict(num_pages=0), INVALID
        yield name, form, dict(num_pages=1 << 27), INVALID
        if form in ("tree", "append"):
            yield name, form, dict(total_q=-1), INVALID
        if form == "append":
            yield name, form, dict(total_q=(1 << 28) + 1), UNSUPPORTED
        if form == "tree":
            yield name, form, dict(max_q=-1), INVALID
            yield name, form, dict(max_q=65), UNSUPPORTED
            yield name, form, dict(max_seq_len=-1), INVALID
            yield name, form, dict(max_seq_len=70 * 16 + 1), INVALID
            yield name, form, dict(max_blocks=20000, max_seq_len=262145), UNSUPPORTED
            yield name, form, dict(out_dtype=2), INVALID
            for splits in (-1, 1, 15, 1025):
                yield name, form, dict(num_splits=splits), INVALID
            yield name, form, dict(ws=None), None
            yield name, form, dict(ws_bytes=16), None
            if kind == "sliding":
                yield name, form, dict(window=0), INVALID
        if form == "commit":
            yield name, form, dict(layers=0), INVALID
            yield name, form, dict(layers=65), UNSUPPORTED
            yield name, form, dict(max_path=0), INVALID
            yield name, form, dict(max_path=65), UNSUPPORTED
            yield name, form, dict(ks=Pools([FAKE, None])), INVALID
            yield name, form, dict(vs=Pools([FAKE + 8, 5 * FAKE])), INVALID
            yield name, form, dict(vs=Pools([3 * FAKE, FAKE])), INVALID  # a pool twice


@pytest.mark.parametrize("name,form,bad,code", list(bad_calls()), ids=lambda x: str(x))
def test_bad_arguments_are_refused_before_launch(lib, name, form, bad, code):
    want = {code} if code is not None else {WORKSPACE, 4}  # (the workspace needs a device to be judged)
    assert call(lib, name, form, **bad) in want
    assert code is None or name in pda.attn_last_error()
    h = ctypes.c_void_p()
    assert lib.attn_step_create(ctypes.byref(h)) == 0
    try:
        assert call(lib, name, form, step=h, **bad) in want
        assert lib.attn_step_num_calls(h) == 0
    finally:
        lib.attn_step_destroy(h)


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_a_commit_writes_none_of_its_inputs(lib, kind):
    name = "attn_kv_commit_" + kind
    sizes = dict(table=4 * 70 * 4, lens=4 * 4, cu_q=4 * 5, path=4 * 8 * 4, path_len=4 * 4)
    apart = {a: (20 + i) * FAKE for i, a in enumerate(sizes)}
    h = ctypes.c_void_p()
    assert lib.attn_step_create(ctypes.byref(h)) == 0
    try:
        for a, n in sizes.items():
            for at in (apart[a], apart[a] - 12, apart[a] + n - 4):
                assert call(lib, name, "commit", step=h, new_lens=at, **apart) == INVALID
                assert "overlaps" in pda.attn_last_error()
        assert lib.attn_step_num_calls(h) == 0
        for a, n in sizes.items():
            for at in (apart[a] - 16, apart[a] + n):
                assert call(lib, name, "commit", step=h, new_lens=at, **apart) == 0
    finally:
        lib.attn_step_destroy(h)


def test_headers_compile_as_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "attn_tree.h"\n#include "attn_step.h"\nint main(void){return ATTN_MAX_TREE - 64;}\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", str(src), "-o",
                    str(tmp_path / "use.o")], check=True)


def test_the_binding_checks_its_tensors(lib):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA tensor"):
        pda.attn_decode_sliding_tree(bf(3, 16, 256), bf(2, 16, 8, 256), bf(2, 16, 8, 256), i32(1, 2), i32(1), i32(2), i32(3))
    with pytest.raises(ValueError, match="q must be"):
        pda.attn_decode_global_tree(bf(3, 16), bf(2, 16, 1, 512), bf(2, 16, 1, 512), i32(1, 2), i32(1), i32(2), i32(3))
    with pytest.raises(ValueError, match="one pool per layer"):
        pda.attn_kv_commit_global([], [], i32(1, 2), i32(1), i32(2), i32(1, 4), i32(1))
    with pytest.raises(ValueError, match="free_list"):
        pda.attn_pages_assign(i32(1), i32(1), i32(1, 2), i32(1, 2), i32(1, 2), i32(2))


def test_tree_plan(lib):
    S, G = pda.KIND_SLIDING, pda.KIND_GLOBAL

    def a256(x):
        return (x + 255) // 256 * 256

    def workspace(grid, rows, D):
        return a256(2 * grid * rows * D * 4) + a256(2 * grid * rows * 8) + a256(grid * 16)

    # long sequences: a block per SM, cut sequences merged by a second kernel; global trees of more than four nodes take
    # pairs of blocks, sliding ones as many rows as hold the longest tree
    assert pda.attn_decode_tree_plan(G, 16, 4, 131072, 0) == (152, 2, workspace(152, 64, 512))
    assert pda.attn_decode_tree_plan(G, 16, 8, 131072, 0) == (152, 2, workspace(152, 64, 512))
    for max_q, rows in ((1, 32), (16, 32), (17, 64), (32, 64), (33, 128), (64, 128)):
        assert pda.attn_decode_tree_plan(S, 64, max_q, 32768, 1024) == (152, 2, workspace(152, rows, 256))
    # one page each, by the caller's bound: the lengths may be longer, and then sequences are cut
    for max_seq_len in (0, 1, 16):
        assert pda.attn_decode_tree_plan(G, 200, 4, max_seq_len, 0) == (152, 2, workspace(152, 64, 512))
    # a few short sequences: a block (or pair) for each group of nodes
    assert pda.attn_decode_tree_plan(G, 3, 4, 256, 0) == (3, 1, a256(3 * 16))
    assert pda.attn_decode_tree_plan(G, 3, 9, 256, 0) == (12, 1, a256(12 * 16))
    assert pda.attn_decode_tree_plan(S, 2, 9, 240, 1024) == (16, 1, a256(16 * 16))
    # forced
    assert pda.attn_decode_tree_plan(G, 1, 1, 200, 0, 16)[0] == 16
    for bad in (dict(kind=2), dict(batch=0), dict(batch=257), dict(max_q=-1), dict(max_q=65), dict(max_seq_len=-1),
                dict(max_seq_len=262145), dict(num_splits=-1), dict(num_splits=3), dict(num_splits=1025),
                dict(num_sms=0)):
        kw = dict(dict(kind=G, batch=1, max_q=4, max_seq_len=100, window=0, num_splits=0, num_sms=152), **bad)
        with pytest.raises(pda.AttnDecodeError):
            pda.attn_decode_tree_plan(**kw)
    # the largest windows and lengths do not overflow
    for w in (2 ** 31 - 1, 262144, 1):
        assert pda.attn_decode_tree_plan(S, 256, 64, 262144, w)[0] == 152
