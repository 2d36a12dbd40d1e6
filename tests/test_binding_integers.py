"""Integers past 32 bits that are no tensor's size (layouts, rules, kinds, groups of experts): the C side takes
int32, and one that is cut to 32 bits on the way would be another call, with buffers checked for the first."""
import inspect

import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
import test_binding_types
import test_mxfp8_ops_refusals
from stand_in import install


@pytest.fixture
def lib(monkeypatch):
    return install(monkeypatch)


def calls():
    return {**test_binding_types.calls(), **test_mxfp8_ops_refusals.calls()}


def integers(f, args):
    """name -> value of the integer arguments, given or by default."""
    out = {}
    for name, p in inspect.signature(f).parameters.items():
        v = args.get(name, p.default)
        if isinstance(v, int) and not isinstance(v, bool):
            out[name] = v
    return out


def test_every_call_is_looked_at():
    assert set(calls()) == {"moe_dispatch", "moe_dispatch_backward", "moe_combine_weighted", "moe_combine_backward",
                            "moe_quant_mxfp4", "moe_quant_mxfp8", "moe_mxfp4_tile_scales", "moe_grouped_gemm_mxfp4",
                            "moe_grouped_gemm_mxfp8", "moe_route_scores", "moe_route_scores_backward", "moe_rmsnorm",
                            "moe_rmsnorm_backward", "moe_swiglu_mxfp8", "moe_swiglu_mxfp8_backward"}
    f, args = calls()["moe_route_scores"]
    assert set(integers(f, args)) == {"score", "num_groups", "topk_groups", "group_score"}


@pytest.mark.parametrize("name", sorted(calls()))
def test_integers_past_32_bits_are_refused(lib, name):
    f, args = calls()[name]
    f(**args)
    assert len(lib.calls) == 1
    for arg, v in integers(f, args).items():
        for cut in (v + 2 ** 32, v - 2 ** 32, v + 2 ** 63, v + 2 ** 64, v + 2 ** 31):
            with pytest.raises(moe.MoEError):
                f(**dict(args, **{arg: cut}))
    assert len(lib.calls) == 1


def test_without_tensors_or_with_outputs_left_out(lib):
    """Where no tensor's size depends on the integer."""
    past = 2 ** 32
    x, y = torch.zeros(4, 96), torch.zeros(4, 96)
    f, args = calls()["moe_swiglu_mxfp8_backward"]
    i32 = dict(dtype=torch.int32)
    ids, inv, maps = torch.zeros(4, 2, **i32), torch.zeros(8, **i32), torch.zeros(8, **i32)
    none = torch.zeros(0, 32)
    for call in (lambda: moe.moe_rmsnorm(x, None, 1e-6, y=y, sf_layout=past),
                 lambda: moe.moe_rmsnorm(x, None, 1e-6, y=y, scale_rule=past),
                 lambda: f(**dict(args, codes=None, sf=None, sf_layout=past)),
                 lambda: moe.moe_dispatch(None, ids, 8 + past, 0, 8, 1, torch.zeros(8, **i32), torch.zeros(9, **i32),
                                          maps, inv, None),
                 lambda: moe.moe_dispatch_backward(torch.zeros(0, 4), torch.zeros(0, **i32), past + 1, torch.zeros(0, 4)),
                 lambda: moe.moe_quant_mxfp8(none, torch.zeros(0, 32, dtype=torch.uint8),
                                             torch.zeros(0, dtype=torch.uint8), past)):
        with pytest.raises(moe.MoEError):
            call()
    assert not lib.calls


def test_sizing_of_integers_past_32_bits_is_zero(lib):
    for past in (2 ** 31, 2 ** 32, 2 ** 64, -2 ** 32):
        assert moe.moe_mxfp4_scale_bytes(1, 4, 64, moe.MOE_SF_TILED + past) == 0
        assert moe.moe_dispatch_rows_capacity(4, 2 + past, 4, 1) == 0
        assert moe.moe_dispatch_rows_capacity(4, 2, 4 + past, 1) == 0
        assert moe.moe_dispatch_rows_capacity(4, 2, 4, 1 + past) == 0
        assert moe.moe_mxfp4_workspace_size(4 + past, 1, 8, 32) == 0
        assert moe.moe_rmsnorm_workspace_size(1000 + past, 64) == 0
