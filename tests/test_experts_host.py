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
