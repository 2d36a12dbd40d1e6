"""What MXExperts asks of the library and of autograd, with a stand-in in the library's place (on
the CPU; no kernel runs, so values are not looked at)."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
from nvfp4_mixture_experts_gb300.experts import MXExperts
from stand_in import install

T, H, I, E, k = 6, 64, 32, 4, 2


@pytest.fixture
def lib(monkeypatch):
    return install(monkeypatch)


def layer(**kw):
    return MXExperts.from_master(E, 0, torch.randn(E, 2 * I, H), torch.randn(E, H, I), **kw)


def inputs():
    x = torch.randn(T, H, requires_grad=True)
    return x, torch.randint(0, E, (T, k), dtype=torch.int32), torch.rand(T, k, requires_grad=True)


def test_second_derivatives_raise(lib):
    ex, (x, ids, w) = layer(), inputs()
    out = ex(x, ids, w)
    for loss in (out.sum(), out.square().sum()):
        dx, dw = torch.autograd.grad(loss, (x, w), create_graph=True)
        for g in (dx, dw):
            with pytest.raises(RuntimeError, match="second derivatives"):
                (x.sum() + w.sum() + g.square().sum()).backward(retain_graph=True)


def test_first_derivatives_do_not_change_under_create_graph(lib):
    ex, (x, ids, w) = layer(), inputs()
    ex(x, ids, w).sum().backward()
    assert x.grad.shape == x.shape and not x.grad.requires_grad
    assert w.grad.shape == w.shape and not w.grad.requires_grad


def test_every_call_that_can_find_errors_on_the_device_is_lent_the_status_word(lib):
    ex, (x, ids, w) = layer(), inputs()
    del lib.calls[:]
    ex(x, ids, w).sum().backward()
    lent = {"moe_dispatch": [], "moe_grouped_gemm_mxfp4": []}
    for name, args in lib.calls:
        if name in lent:
            lent[name].append(args[-2])          # the argument before the stream
    assert lent == {"moe_dispatch": [ex.status.data_ptr()],
                    "moe_grouped_gemm_mxfp4": [ex.status.data_ptr()] * 4}


@pytest.mark.parametrize("bits,status", [(0, moe.MOE_OK), (moe.MOE_DEV_BAD_EXPERT_ID, moe.MOE_ERR_DEVICE_STATUS),
                                         (moe.MOE_DEV_WAIT_TIMEOUT | moe.MOE_DEV_BAD_INDEX, moe.MOE_ERR_TIMEOUT)])
def test_status_is_read_and_cleared(lib, bits, status):
    ex = layer(backward=False)
    ex.status.fill_(bits)
    assert ex.get_status() == (status, bits)
    assert ex.get_status() == (moe.MOE_OK, 0)


def test_checkpoint_scales_of_another_size_are_refused(lib):
    def parts():
        return [torch.zeros(E, 2 * I, H // 2, dtype=torch.uint8), torch.zeros(E, 2 * I, H // 32, dtype=torch.uint8),
                torch.zeros(E, H, I // 2, dtype=torch.uint8), torch.zeros(E, H, I // 32, dtype=torch.uint8)]

    MXExperts.from_checkpoint(E, 0, *parts())
    for i in (1, 3):
        bad = parts()
        bad[i] = bad[i][:, 1:].contiguous()
        with pytest.raises(moe.MoEError):
            MXExperts.from_checkpoint(E, 0, *bad)
