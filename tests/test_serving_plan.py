"""The decodes' launch plans on devices of other sizes and at the ends of their arguments' range."""

import pytest
import torch

import paged_decode_attention_gb300 as pda
from paged_decode_attention_gb300 import _build
from workloads import make_case

from _fp8 import Fp8Case


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return pda.load()


@pytest.mark.parametrize("num_sms", [8, 76, 132, 152, 304])
def test_short_sliding_sequences_get_a_block_each_while_their_blocks_are_resident(num_sms):
    # three blocks per SM, eight KV heads: one wave
    wave = num_sms * 3 // 8
    for batch in sorted({1, wave, min(256, wave + 1)}):
        blocks, launches, _ = pda.attn_decode_fp8_plan(pda.KIND_SLIDING, batch, 128, 1024, 0, num_sms)
        if batch <= wave:
            assert (blocks, launches) == (batch, 1)
        else:
            assert blocks == wave


TOP = 2 ** 31 - 1


@pytest.mark.parametrize("kind", [pda.KIND_SLIDING, pda.KIND_GLOBAL])
@pytest.mark.parametrize("batch", [1, 4, 256])
def test_the_largest_window_is_none(kind, batch):
    for longest in (100, 5000, 262144):
        none = 1 << 24  # as wide, for every length
        assert pda.attn_decode_fp8_plan(kind, batch, longest, TOP) == pda.attn_decode_fp8_plan(kind, batch, longest, none)
        assert pda.attn_decode_plan(kind, batch, longest, TOP) == pda.attn_decode_plan(kind, batch, longest, none)
        assert pda.attn_decode_launches(kind, batch, longest, TOP) == pda.attn_decode_launches(kind, batch, longest, none)


@pytest.mark.parametrize("batch", [1, 4, 256])
def test_the_largest_length_is_long(batch):
    # (beyond what the calls take; a window caps the pages, and without one the blocks are all the device's)
    for plan in (pda.attn_decode_fp8_plan, pda.attn_decode_plan, pda.attn_decode_launches):
        assert plan(pda.KIND_SLIDING, batch, TOP, 1024) == plan(pda.KIND_SLIDING, batch, 262144, 1024)
        assert plan(pda.KIND_GLOBAL, batch, TOP, 0) == plan(pda.KIND_GLOBAL, batch, 262144, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["sliding", "global", "sliding_fp8", "global_fp8"])
def test_a_call_with_the_largest_window_sees_everything(cuda_lib, name):
    case = make_case(name.split("_")[0], [3, 700, 5000, 0], seed=110, window=0)
    if name.endswith("fp8"):
        args = Fp8Case(case).on("cuda:0")
    else:
        c = case.to("cuda:0")
        args = (c.q, c.k_pool, c.v_pool, c.block_table, c.seq_lens)
    fn = getattr(pda, "attn_decode_" + name)
    st = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    a, b = (fn(*args, window=w, out_dtype=torch.float32, status=st) for w in (TOP, 1 << 24))
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.isfinite(a).all() and torch.equal(a, b)
