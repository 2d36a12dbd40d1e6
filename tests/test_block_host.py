"""What the 8-bit experts, the shared expert and the block ask of the library, with a stand-in in the
library's place (on the CPU; no kernel runs, so values are not looked at)."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
from nvfp4_mixture_experts_gb300.block import MXBlock, rms_norm, route
from nvfp4_mixture_experts_gb300.experts import MXExperts, MXShared
from stand_in import install

T, H, I, E, k = 6, 128, 128, 4, 2


@pytest.fixture
def lib(monkeypatch):
    return install(monkeypatch)


def experts(**kw):
    return MXExperts.from_master(E, 0, torch.randn(E, 2 * I, H), torch.randn(E, H, I), act_bits=8, **kw)


def shared():
    return MXShared.from_master(torch.randn(1, 2 * I, H), torch.randn(1, H, I))


def names(lib):
    return [c[0] for c in lib.calls]


def test_calls_of_the_experts(lib):
    ex = experts()
    x, w = torch.randn(T, H, requires_grad=True), torch.rand(T, k, requires_grad=True)
    ids = torch.randint(0, E, (T, k), dtype=torch.int32)
    del lib.calls[:]
    out = ex(x, ids, w)
    assert names(lib) == ["moe_dispatch", "moe_quant_mxfp8", "moe_grouped_gemm_mxfp8", "moe_swiglu_mxfp8",
                          "moe_grouped_gemm_mxfp8", "moe_combine_weighted"]
    assert lib.calls[3][1][-3] is not None            # a checkpoint is kept
    del lib.calls[:]
    out.sum().backward()
    assert names(lib) == ["moe_combine_backward", "moe_quant_mxfp8", "moe_grouped_gemm_mxfp8",
                          "moe_swiglu_mxfp8_backward", "moe_grouped_gemm_mxfp8", "moe_dispatch_backward"]
    for name, args in lib.calls:
        if name == "moe_grouped_gemm_mxfp8":
            assert args[-2] == ex.status.data_ptr()
    del lib.calls[:]
    ex(x.detach(), ids, w.detach())
    assert lib.calls[3][0] == "moe_swiglu_mxfp8" and lib.calls[3][1][-3] is None   # nothing is kept


def test_sizes_and_bits_that_do_not_fit(lib):
    for h, i, bits in ((64, 128, 8), (128, 64, 8), (128, 128, 6)):
        with pytest.raises(moe.MoEError):
            MXExperts.from_master(E, 0, torch.randn(E, 2 * i, h), torch.randn(E, h, i), act_bits=bits)
    with pytest.raises(moe.MoEError):
        MXShared.from_master(torch.randn(2, 2 * I, H), torch.randn(2, H, I))
    with pytest.raises(moe.MoEError):   # the codes of other rows
        shared()(torch.randn(T, H), (torch.zeros(T - 1, H, dtype=torch.uint8), torch.zeros(2048, dtype=torch.uint8)))


def test_no_backward_without_transposed_weights(lib):
    x = torch.randn(T, H, requires_grad=True)
    ids = torch.randint(0, E, (T, k), dtype=torch.int32)
    with pytest.raises(RuntimeError):
        experts(backward=False)(x, ids, torch.rand(T, k)).sum().backward()
    with pytest.raises(RuntimeError):
        MXShared.from_master(torch.randn(1, 2 * I, H), torch.randn(1, H, I), backward=False)(x).sum().backward()


def test_second_derivatives_raise(lib):
    x = torch.randn(T, H, requires_grad=True)
    dx, = torch.autograd.grad(shared()(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        dx.sum().backward()
    w, r = torch.rand(H, requires_grad=True), torch.randn(T, H)
    y, h, _, _ = rms_norm(x, w, residual=r)
    for g in torch.autograd.grad(y.sum() + h.sum(), (x, w), create_graph=True):
        with pytest.raises(RuntimeError, match="second derivatives"):
            g.sum().backward(retain_graph=True)
    _, wt = route(x, 3)
    dx, = torch.autograd.grad(wt.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        dx.sum().backward()


def test_block(lib):
    norm, router = torch.ones(H, requires_grad=True), torch.randn(E, H, requires_grad=True)
    bl = MXBlock(norm, router, experts(), k, shared=shared(), score=moe.MOE_SCORE_SIGMOID, num_groups=2)
    x, r = torch.randn(T, H, requires_grad=True), torch.randn(T, H, requires_grad=True)
    del lib.calls[:]
    out, h = bl(x, r)
    assert names(lib)[:2] == ["moe_rmsnorm", "moe_route_scores"]
    # the shared expert reads the norm's own 8-bit rows
    assert names(lib).count("moe_quant_mxfp8") == 1
    (out.sum() + h.sum()).backward()
    assert names(lib)[-1] == "moe_rmsnorm_backward" and "moe_route_scores_backward" in names(lib)
    for t in (x, r, norm, router):
        assert t.grad.shape == t.shape
    bl.shared.status.fill_(moe.MOE_DEV_BAD_INDEX)
    assert bl.get_status() == (moe.MOE_ERR_DEVICE_STATUS, moe.MOE_DEV_BAD_INDEX)
    bl.experts.status.fill_(moe.MOE_DEV_WAIT_TIMEOUT)
    assert bl.get_status() == (moe.MOE_ERR_TIMEOUT, moe.MOE_DEV_WAIT_TIMEOUT)
    assert bl.get_status() == (moe.MOE_OK, 0)


def test_gradients_of_unused_results(lib):
    x, r = torch.randn(T, H, requires_grad=True), torch.randn(T, H, requires_grad=True)
    _, h, _, _ = rms_norm(x, torch.ones(H), residual=r)
    h.sum().backward()
    assert names(lib)[-1] == "moe_rmsnorm_backward" and x.grad.shape == r.grad.shape == (T, H)
    y, h, codes, sf = rms_norm(x, torch.ones(H), eight=True)
    assert h is x and not codes.requires_grad and not sf.requires_grad


def strides(lib, name):
    """The row strides that the calls of this name were given."""
    at = {"moe_rmsnorm": (2, 4), "moe_rmsnorm_backward": (2, 4), "moe_route_scores": (2,), "moe_quant_mxfp8": (5,)}
    return [args[i] for call, args in lib.calls if call == name for i in at[name]]


def test_rows_that_repeat_or_are_transposed(lib):
    """Gradients and inputs that are broadcast over the tokens (row stride 0) or transposed."""
    x, r = torch.randn(T, H, requires_grad=True), torch.randn(1, H, requires_grad=True)
    y, h, _, _ = rms_norm(x, torch.ones(H), residual=r.expand(T, H))
    (y.sum(0) * torch.rand(H)).sum().backward(retain_graph=True)     # dy, dh: one row for all tokens
    (y.sum(0) * torch.rand(H) + h.sum(0) * torch.rand(H)).sum().backward()
    assert r.grad.shape == (1, H) and all(s in (0, H) for s in strides(lib, "moe_rmsnorm_backward"))
    rms_norm(torch.randn(H).expand(T, H), torch.ones(H))
    rms_norm(torch.randn(H, T).t(), torch.ones(H))
    route(torch.randn(H).expand(T, H), k)
    route(torch.randn(H, T).t(), k)
    sh = shared()
    for a in (torch.randn(H).expand(T, H), torch.randn(H, T).t(), torch.randn(T, 2 * H)[:, :H]):
        sh(a)
    assert strides(lib, "moe_rmsnorm") == [H, H, H, 0, H, 0]
    assert strides(lib, "moe_route_scores") == [H, H]
    assert strides(lib, "moe_quant_mxfp8")[-3:] == [H, H, 2 * H]
    # of dy and dh a row's stride is the rows' own
    back = [args for call, args in lib.calls if call == "moe_rmsnorm_backward"]
    assert [a[2] for a in back] == [H, H] and back[1][4] == H
