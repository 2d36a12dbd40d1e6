"""Sizes next to the largest 32-bit number: counts that are rounded up on the way to a launch or in a
kernel must not pass it."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


def test_one_pair_a_token_of_the_most_tokens():
    inv = torch.full((MOST,), -1, dtype=torch.int32, device="cuda")
    rows = torch.tensor([[3.0], [5.0]], dtype=torch.bfloat16, device="cuda")
    inv[0], inv[MOST - 1] = 0, 1
    dx = torch.full((MOST, 1), -3.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_dispatch_backward(rows, inv, 1, dx)
    assert dx[0].item() == 3.0 and dx[MOST - 1].item() == 5.0
    dx[0], dx[MOST - 1] = 0, 0
    assert not torch.any(dx)


def test_product_of_the_most_rows():
    a = torch.zeros(MOST, 16, dtype=torch.uint8, device="cuda")
    a[MOST - 2:] = 0x22                                             # ones
    sf = torch.full((moe.moe_mxfp4_scale_bytes(1, MOST, 32, moe.MOE_SF_TILED),), 127, dtype=torch.uint8, device="cuda")
    w = torch.full((1, 1, 16), 0x44, dtype=torch.uint8, device="cuda")   # twos
    wsf = torch.full((512,), 127, dtype=torch.uint8, device="cuda")
    out = torch.full((MOST, 1), -3.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_grouped_gemm_mxfp4(a, sf, None, None, w, wsf, out, status=status)
    assert status.item() == 0
    assert torch.all(out[MOST - 2:] == 64.0) and torch.all(out[:4096] == 0.0)
    out[MOST - 2:] = 0
    assert not torch.any(out)
