"""A NaN at a visible position of a bf16 cache shows in the outputs that it belongs to, and in no others, however the
sequences are cut into blocks (attn_decode_sliding, attn_decode_global, attn_decode_global_shared)."""

import pytest
import torch

import paged_decode_attention_gb300 as pda
from workloads import key_weight, make_case

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAMES = ["sliding", "global", "global_shared"]


def decode(name, case, num_splits):
    c = case.to(DEV)
    pools = (c.v_pool, key_weight(512, 97, device=DEV)) if name == "global_shared" else (c.k_pool, c.v_pool)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    o = getattr(pda, "attn_decode_" + name)(c.q, *pools, c.block_table, c.seq_lens, window=c.window,
                                            max_seq_len=c.max_seq_len, num_splits=num_splits, out_dtype=torch.float32,
                                            status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return o


def with_nan(case, pool, page, row, head, dims):
    keep = pool[page, row, head].clone()
    pool[page, row, head, dims] = float("nan")
    return keep


@pytest.mark.parametrize("num_splits", [0, 1, 7, 40])
@pytest.mark.parametrize("name", NAMES)
def test_a_visible_nan_shows_and_stays_in_its_sequence(cuda_lib, name, num_splits):
    case = make_case(name.split("_")[0], [500, 500, 700, 0], seed=96)
    clean = decode(name, case, num_splits)
    assert torch.isfinite(clean).all()
    G = 16 // case.k_pool.shape[2]
    page, row = int(case.block_table[1, 20]), 3
    for what, pool in (("key", case.k_pool), ("value", case.v_pool)):
        if name == "global_shared" and what == "key":
            continue
        # a key whole, a value in one dim (of a values-only cache, the key with it)
        keep = with_nan(case, pool, page, row, 0, slice(None) if what == "key" else 9)
        o = decode(name, case, num_splits)
        pool[page, row, 0] = keep
        hit = o[1, :G]
        assert torch.isnan(hit[..., 9] if what == "value" and name != "global_shared" else hit).all(), what
        if what == "value" and name != "global_shared":
            hit[..., 9] = clean[1, :G, 9]
            assert torch.equal(hit, clean[1, :G])
        o[1, :G] = clean[1, :G]
        assert torch.equal(o, clean), what


@pytest.mark.parametrize("num_splits", [0, 1, 40])
@pytest.mark.parametrize("name", NAMES)
def test_nothing_but_nan_is_visible(cuda_lib, name, num_splits):
    # one position; a page of which every row is NaN; pages of them, cut between blocks
    for n in (1, 16, 300):
        case = make_case(name.split("_")[0], [n, 20], seed=98)
        clean = decode(name, case, num_splits)
        for p in range(-(-n // 16)):
            case.k_pool[int(case.block_table[0, p])] = float("nan")
            if name == "global_shared":
                case.v_pool[int(case.block_table[0, p])] = float("nan")
        o = decode(name, case, num_splits)
        assert torch.isnan(o[0]).all(), n
        assert torch.equal(o[1], clean[1]), n
