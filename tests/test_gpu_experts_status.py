"""Errors that MXExperts' calls find on the device."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
from nvfp4_mixture_experts_gb300.experts import MXExperts


@pytest.mark.gpu
@pytest.mark.parametrize("T", [9, 700])
def test_an_expert_id_out_of_range_shows_in_the_status(T):
    torch.manual_seed(T)
    E, H, I, k = 4, 64, 32, 2
    ex = MXExperts.from_master(E, 0, torch.randn(E, 2 * I, H, device="cuda"),
                               torch.randn(E, H, I, device="cuda"))
    x = torch.randn(T, H, device="cuda", requires_grad=True)
    ids = torch.randint(0, E, (T, k), device="cuda", dtype=torch.int32)
    w = torch.rand(T, k, device="cuda")
    good = ex(x, ids, w)
    good.sum().backward()
    assert ex.get_status() == (moe.MOE_OK, 0)
    ids[T // 2, 1] = E
    out = ex(x, ids, w)
    assert ex.get_status() == (moe.MOE_ERR_DEVICE_STATUS, moe.MOE_DEV_BAD_EXPERT_ID)
    others = torch.arange(T, device="cuda") != T // 2
    assert torch.equal(out[others], good[others]) and not torch.equal(out[~others], good[~others])
    assert ex.get_status() == (moe.MOE_OK, 0)
