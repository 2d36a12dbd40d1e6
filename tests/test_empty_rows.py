"""Sorted rows of no capacity have nothing to write (answered on the host)."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
from stand_in import install
from test_ops_refusals import BACK, call, lib  # noqa: F401


def test_a_gradient_of_rows_of_no_capacity_is_nothing(lib):  # noqa: F811
    assert call(lib, "moe_combine_backward", BACK, cap=0, y=None, dy=None, dw=None) == moe.MOE_OK


def test_the_binding_wants_one_of_the_two_gradients(monkeypatch):
    s = install(monkeypatch)
    x, inv, w = torch.zeros(4, 8), torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2)
    for y in (None, torch.zeros(8, 8)):
        with pytest.raises(moe.MoEError):
            moe.moe_combine_backward(x, y, inv, w, None, None)
    assert not s.calls


def test_more_pairs_a_token_than_rows_can_be_sized_for(monkeypatch):
    from nvfp4_mixture_experts_gb300.experts import MXExperts
    install(monkeypatch)
    E, H = 40, 32
    ex = MXExperts.from_master(E, 0, torch.randn(E, 64, H), torch.randn(E, H, 32), backward=False)
    with pytest.raises(moe.MoEError):
        ex(torch.randn(5, H), torch.zeros(5, 33, dtype=torch.int32), torch.rand(5, 33))
