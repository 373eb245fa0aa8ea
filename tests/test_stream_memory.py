"""Calls on another stream than the one that their memory comes from.

A call's output and workspace, where it makes them itself, must be filled before its kernels read them and must not be
handed out again while its kernels write them, whichever stream the call is on.  One of the two streams is held back by
kernels that take a millisecond each, so that what is ordered by nothing but luck comes in the wrong order."""

import dataclasses

import pytest
import torch

import paged_decode_attention_gb300 as pda
from workloads import key_weight, make_append_case, make_case

from _fp8 import Fp8Case
from test_chunk_append import Chunk
from test_prefix_decode import Case as PrefixCase

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
LENS = [5, 700, 1300, 64]


@dataclasses.dataclass
class Call:
    name: str        # attn_<name>, prepare_<name>, Step.add_<name>
    args: list
    kw: dict
    workspace: int   # bytes it makes for itself, 0: none


def decode_call(name):
    kind = "sliding" if "sliding" in name else "global"
    const = getattr(pda, "KIND_" + kind.upper())
    window = 1024 if kind == "sliding" else 0
    kw = dict(window=window, max_seq_len=1300, out_dtype=torch.float32)
    case = make_case(kind, LENS, seed=90)
    if name.endswith("_fp8"):
        return Call(name, list(Fp8Case(case).on(DEV)), kw, pda.attn_decode_fp8_workspace_size(const, 4, 1300, window))
    c = case.to(DEV)
    pools = [c.v_pool, key_weight(512, 91, device=DEV)] if name.endswith("_shared") else [c.k_pool, c.v_pool]
    return Call(name, [c.q] + pools + [c.block_table, c.seq_lens], kw,
                pda.attn_decode_workspace_size(const, 4, 1300, window))


def prefix_call(name):
    return Call(name, PrefixCase(1000, LENS, seed=92).args(), dict(max_seq_len=1300, prefix_splits=2,
                                                                   out_dtype=torch.float32),
                pda.attn_decode_prefix_workspace_size(4, 1008, 1300, 0, 2))


def append_call(name):
    kind = "sliding" if "sliding" in name else "global"
    if name.endswith(("_chunk", "_fp8")):
        c = Chunk(kind, [40, 3, 90], [8, 3, 1], 93)
        return Call(name, c.common() + list(c.bf16_pools() if name.endswith("_chunk") else c.fp8_cache()), {}, 0)
    a = make_append_case(kind, [0, 16, 333], seed=94, full_cache=True).to(DEV)
    return Call(name, [a.qkv, a.w_q, a.w_k, a.cache.block_table, a.positions, a.cache.k_pool, a.cache.v_pool], {}, 0)


def prefill_call(name):
    kind = "sliding" if "sliding" in name else "global"
    c = make_case(kind, [40, 700], seed=95).to(DEV)
    g = torch.Generator().manual_seed(95)
    q = torch.randn((43, c.Hq, c.D), generator=g).to(torch.bfloat16).to(DEV)
    cu = torch.tensor([0, 40, 43], dtype=torch.int32, device=DEV)
    return Call(name, [q, c.k_pool, c.v_pool, c.block_table, c.seq_lens, cu], dict(max_q=40), 0)


DECODES = ["decode_sliding", "decode_global", "decode_global_shared", "decode_sliding_fp8", "decode_global_fp8"]
APPENDS = ["kv_append_%s%s" % (k, f) for k in ("sliding", "global") for f in ("", "_chunk", "_fp8")]
PREFILLS = ["prefill_sliding", "prefill_global"]


def make(name):
    build = prefix_call if "prefix" in name else prefill_call if "prefill" in name else \
        append_call if "append" in name else decode_call
    return build(name)


def hold(stream, milliseconds=40):
    a, b = (torch.zeros(4, dtype=torch.int32, device=DEV) for _ in range(2))
    torch.cuda.synchronize()
    for _ in range(milliseconds):
        pda.selftest_delayed_copy(a, b, delay_ns=1000000, stream=stream)
    return a, b  # (kept by the caller until its work is done)


def leave_garbage(nbytes):
    """The next block of this size on the current stream is not zero."""
    if nbytes:
        x = torch.full((nbytes,), 0x7f, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        del x


def expected(c, fn):
    out = fn(*c.args, **c.kw)
    torch.cuda.synchronize()
    return out.clone()


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", DECODES + ["decode_global_prefix"] + APPENDS + PREFILLS)
def test_one_shot_on_a_side_stream_while_the_current_one_is_held(cuda_lib, name, raw):
    c = make(name)
    fn = getattr(pda, "attn_" + name)
    want = expected(c, fn)
    side = torch.cuda.Stream()
    leave_garbage(c.workspace)
    held = hold(torch.cuda.current_stream())
    out = fn(*c.args, stream=side.cuda_stream if raw else side, **c.kw)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del held


@pytest.mark.parametrize("name", DECODES + ["decode_global_prefix"] + APPENDS + PREFILLS)
def test_memory_of_a_held_one_shot_is_not_handed_out(cuda_lib, name):
    # the call waits on its stream; the current stream meanwhile takes and fills blocks of the sizes that it uses
    c = make(name)
    fn = getattr(pda, "attn_" + name)
    want = expected(c, fn)
    side = torch.cuda.Stream()
    torch.cuda.empty_cache()
    held = hold(side)
    out = fn(*c.args, stream=side, **c.kw)
    sizes = [s for s in (c.workspace, want.numel() * want.element_size()) if s]
    taken = [torch.full((s,), 0x55, dtype=torch.uint8, device=DEV) for s in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for x in taken:
        assert (x == 0x55).all()
    del held


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", DECODES + ["decode_global_prefix", "kv_append_global_chunk", "kv_append_sliding_fp8"])
def test_first_run_of_a_prepared_call_on_a_side_stream(cuda_lib, name, raw):
    c = make(name)
    want = expected(c, getattr(pda, "attn_" + name))
    side = torch.cuda.Stream()
    leave_garbage(c.workspace)
    held = hold(torch.cuda.current_stream())
    call = getattr(pda, "prepare_" + name)(*c.args, **c.kw)
    handle = side.cuda_stream if raw else side
    for _ in range(2):
        out = call.run(handle)
        side.synchronize()
        assert torch.equal(out, want)
        with torch.cuda.stream(side):
            out.fill_(7)
    torch.cuda.synchronize()
    call.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del held


@pytest.mark.parametrize("mode", ["graph", "direct"])
def test_first_launch_of_a_step_on_a_side_stream(cuda_lib, mode):
    calls = [make(n) for n in DECODES + ["decode_global_prefix", "kv_append_global_chunk"]]
    wants = [expected(c, getattr(pda, "attn_" + c.name)) for c in calls]
    side = torch.cuda.Stream()
    for c in calls:
        leave_garbage(c.workspace)
    held = hold(torch.cuda.current_stream())
    step = pda.Step()
    outs = [getattr(step, "add_" + c.name)(*c.args, **c.kw) for c in calls]
    step.finalize(mode)
    step.launch(side)
    side.synchronize()
    for o, w in zip(outs, wants):
        assert torch.equal(o, w)
    step.close()
    del held


def test_memory_of_a_dropped_prepared_call_is_not_handed_out_under_its_run(cuda_lib):
    c = make("decode_global_fp8")
    want = expected(c, pda.attn_decode_global_fp8)
    side = torch.cuda.Stream()
    torch.cuda.empty_cache()
    call = pda.prepare_decode_global_fp8(*c.args, **c.kw)
    held = hold(side)
    out = call.run(side)
    del call
    taken = [torch.full((c.workspace,), 0x55, dtype=torch.uint8, device=DEV) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for x in taken:
        assert (x == 0x55).all()
    del held


def test_a_run_captured_before_any_other(cuda_lib):
    # the capture waits for nothing; an eager run on a third stream comes after it
    c = make("decode_sliding_fp8")
    want = expected(c, pda.attn_decode_sliding_fp8)
    call = pda.prepare_decode_sliding_fp8(*c.args, **c.kw)
    side, third = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = call.run(side)
    for go in (graph.replay, lambda: call.run(third)):
        out.fill_(7)
        torch.cuda.synchronize()
        go()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_a_call_prepared_inside_a_capture(cuda_lib):
    # its workspace is zeroed by every replay
    c = make("decode_sliding_fp8")
    want = expected(c, pda.attn_decode_sliding_fp8)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call = pda.prepare_decode_sliding_fp8(*c.args, **c.kw)
        out = call.run()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        out.fill_(7)
