"""Chunk appends on lengths that do not fit together and on rows at the ends of the input's range."""

import numpy as np
import pytest
import torch

import paged_decode_attention_gb300 as pda

from test_chunk_append import Chunk, check_chunk, check_fp8, run_chunk, run_fp8

pytestmark = pytest.mark.gpu


# In the first table four ends (7, 8, 18, 0) lie at or before the last packed row, 19, which a count of ends takes for row
# 19 - 18 of the fifth sequence: position 32 - (0 - 18) + (19 - 18) = 51 of a table of 32.
DECREASING = [([0, 7, 20, 8, 18, 0], [1, 15, 30, 12, 32]), ([0, 9, 3, 4, 20], [9, 32, 8, 16]),
              ([0, 20, 19], [20, 32]), ([5, 0], [32]), ([0, -1, 20], [32, 32])]


@pytest.mark.parametrize("cu,lens", DECREASING, ids=str)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_a_decreasing_cu_q_is_flagged_and_nothing_is_written(cuda_lib, kind, fp8, cu, lens):
    c = Chunk(kind, [20], [20], seed=80, extra_pages=2 * len(lens))
    c.L = lens
    c.cu = torch.tensor(cu, dtype=torch.int32)
    c.table = torch.arange(2 * len(lens), dtype=torch.int32).view(-1, 2)  # every page of 32 positions a sequence
    if fp8:
        q, (k, v, ks, vs), st = run_fp8(c)
        assert (k.view(torch.uint8) == 0x11).all() and (v.view(torch.uint8) == 0x92).all()
        assert (ks.view(torch.uint8) == 120).all() and (vs.view(torch.uint8) == 131).all()
    else:
        q, k, v, st = run_chunk(c)
        assert (k == 3.0).all() and (v == -5.0).all()
    assert st == pda.DEV_BAD_SEQ_LEN and (q == 7.0).all()


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_equal_ends_are_no_decrease(cuda_lib, kind):
    # sequences without new tokens at the start, in a row and at the end
    new = [0, 0, 3, 0, 0, 0, 17, 0]
    c = Chunk(kind, [4, 0, 9, 0, 31, 2, 40, 0], new, seed=81)
    q, k, v, st = run_chunk(c)
    assert st == 0 and not (q == 7.0).all(-1).any()
    assert np.isfinite(k.double().cpu().numpy()[c.page, c.row]).all()


@pytest.mark.parametrize("exponent", [57, 60, 64, 90, 120, 125])
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_rows_whose_squares_leave_the_range_of_fp32(cuda_lib, kind, exponent):
    # (sum x^2 passes 2^128 from a root mean square of 2^60 (D = 256) or 2^59.5 (D = 512) on)
    check_chunk(Chunk(kind, [40, 7], [9, 7], 82, scale=2.0 ** exponent))
    check_fp8(Chunk(kind, [40, 7], [9, 7], 83, scale=2.0 ** exponent))


@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_one_element_at_the_top_of_the_range(cuda_lib, kind):
    # one element of every head row dominates all others, up to the largest bf16
    for value in (2.0 ** 64, -(2.0 ** 100), float(torch.finfo(torch.bfloat16).max)):
        c = Chunk(kind, [40, 7], [9, 7], 84)
        c.qkv.view(c.qkv.shape[0], -1, c.D)[:, :, 5] = value
        check_chunk(c)
        check_fp8(c)
