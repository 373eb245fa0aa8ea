"""The launch plans of the 8-bit decode on devices of other sizes, as host arithmetic."""

import pytest

import paged_decode_attention_gb300 as pda
from paged_decode_attention_gb300 import _build


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
