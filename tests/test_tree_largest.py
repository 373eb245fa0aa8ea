"""The tree attention's plan for any number of splits, and its schedule at the largest batch, trees and lengths."""

import pytest
import torch

import paged_decode_attention_gb300 as pda
from workloads import GLOBAL, PAGE_SIZE, SLIDING

from _fp8 import decode_bound
from _tree import DEV

SHAPE = {"sliding": SLIDING, "global": GLOBAL}


@pytest.mark.parametrize("kind", [pda.KIND_SLIDING, pda.KIND_GLOBAL])
@pytest.mark.parametrize("max_q", [1, 4, 5, 8, 9, 64])
@pytest.mark.parametrize("splits", [16, 17, 41, 151, 1023, 1024])
def test_a_plan_takes_the_splits_it_is_given(kind, max_q, splits):
    window = 1024 if kind == pda.KIND_SLIDING else 0
    assert pda.attn_decode_tree_plan(kind, 3, max_q, 5000, window, splits)[:2] == (splits, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["sliding", "global"])
def test_the_largest_call(cuda_lib, kind):
    """256 sequences of 262144 positions and chains of 64 nodes, all over the same few pages: what every node of one
    sequence sees is known by counting, and all sequences have the same outputs up to where they are cut."""
    sh = SHAPE[kind]
    Hq, Hkv, D = sh["Hq"], sh["Hkv"], sh["D"]
    G, B, n, L = Hq // Hkv, 256, 64, 262144
    ctx, shared = L - n, 8
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((shared + n // PAGE_SIZE, PAGE_SIZE, Hkv, D), generator=g).to(torch.bfloat16) for _ in "kv")
    row = torch.cat([torch.arange(ctx // PAGE_SIZE) % shared, shared + torch.arange(n // PAGE_SIZE)]).to(torch.int32)
    q = (2.5 * torch.randn((n, Hq, D), generator=g) / D ** 0.5).to(torch.bfloat16)
    # a window longer than the table on sliding layers, so that all of it is seen
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o = getattr(pda, "attn_decode_%s_tree" % kind)(
        q.repeat(B, 1, 1).to(DEV), k.to(DEV), v.to(DEV), row[None].repeat(B, 1).to(DEV),
        torch.full((B,), L, dtype=torch.int32, device=DEV), n * torch.arange(B + 1, dtype=torch.int32, device=DEV),
        torch.arange(-1, n - 1, dtype=torch.int32, device=DEV).repeat(B), window=2 * L if kind == "sliding" else 0,
        out_dtype=torch.float32, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    count = torch.cat([torch.bincount(row[:ctx // PAGE_SIZE].long(), minlength=shared).repeat_interleave(PAGE_SIZE),
                       torch.ones(n, dtype=torch.long)]).double()
    seen = torch.cat([torch.ones((n, shared * PAGE_SIZE)), torch.ones((n, n)).tril()], 1).double() * count
    o = o.view(B, n, Hq, D)
    for h in range(Hq):
        kh, vh = k[:, :, h // G].reshape(-1, D).double(), v[:, :, h // G].reshape(-1, D).double()
        w = torch.softmax(q[:, h].double() @ kh.t() + torch.log(seen), -1)
        S = (q[:, h].double().abs() @ kh.abs().t()).max(-1, keepdim=True).values
        want = w @ vh
        bound = decode_bound(want, w @ vh.abs(), S, D, torch.float32, 2.0 ** -8)
        assert ((o[:, :, h].cpu().double() - want).abs() <= bound).all()
