"""A second derivative raises by the name of the operator that has none (a stand-in in the library's place)."""
import pytest
import torch

from nvfp4_mixture_experts_gb300.block import rms_norm, route
from nvfp4_mixture_experts_gb300.experts import MXExperts, MXShared
from stand_in import install

T, H, I, E, k = 6, 128, 128, 4, 2


@pytest.fixture(autouse=True)
def lib(monkeypatch):
    return install(monkeypatch)


def of_experts(x, bits):
    ex = MXExperts.from_master(E, 0, torch.randn(E, 2 * I, H), torch.randn(E, H, I), act_bits=bits)
    return ex(x, torch.zeros(T, k, dtype=torch.int32), torch.rand(T, k))


CASES = [("MXExperts", lambda x: of_experts(x, 4)), ("MXExperts", lambda x: of_experts(x, 8)),
         ("MXShared", lambda x: MXShared.from_master(torch.randn(1, 2 * I, H), torch.randn(1, H, I))(x)),
         ("rms_norm", lambda x: rms_norm(x, torch.ones(H))[0]), ("route", lambda x: route(x, k)[1])]


@pytest.mark.parametrize("name,f", CASES)
def test_the_error_names_the_operator(name, f):
    x = torch.randn(T, H, requires_grad=True)
    dx, = torch.autograd.grad(f(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="^%s has no second derivatives" % name):
        dx.sum().backward()
