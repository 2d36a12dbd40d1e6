"""The experts and the shared expert with 8-bit activations and fp16 tokens: gate, up and the gradient of their
product may be past fp16's largest number, or below its steps, where the results are not."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
from nvfp4_mixture_experts_gb300.experts import MXExperts, MXShared
from test_gpu_block import TOL, four, gated, gated_back, masters, rel

pytestmark = pytest.mark.gpu
UP = [1.0, 2e5, 1e-5]   # of up's weights (the down product's by the inverse): gate_up past 65504; the gradient past it


def weights(E, H, I, up, g):
    w13, w2 = masters(E, H, I, g)
    w13[:, I:] *= up
    return w13, w2 / up


@pytest.mark.parametrize("T,H,I", [(1, 128, 128), (150, 256, 384)])
@pytest.mark.parametrize("up", UP)
def test_shared_expert(T, H, I, up):
    g = torch.Generator("cuda").manual_seed(T)
    w13, w2 = weights(1, H, I, up, g)
    sh = MXShared.from_master(w13, w2)
    x = torch.randn(T, H, generator=g, device="cuda").half().requires_grad_()
    out = sh(x)
    dout = torch.randn(T, H, generator=g, device="cuda").half()
    out.backward(dout)
    y, held = gated(x.detach().cpu(), 0, four(w13), four(w2), I)
    dx = gated_back(dout.cpu(), held, 0, four(w13, True), four(w2, True), I)
    assert out.dtype == x.grad.dtype == torch.float16
    assert rel(out, y) < TOL and rel(x.grad, dx) < TOL


@pytest.mark.parametrize("T,H,I,E,k,off,El", [(1, 128, 128, 4, 2, 0, 4), (37, 256, 128, 8, 3, 2, 5)])
@pytest.mark.parametrize("up", UP)
def test_experts(T, H, I, E, k, off, El, up):
    g = torch.Generator("cuda").manual_seed(T)
    w13, w2 = weights(El, H, I, up, g)
    ex = MXExperts.from_master(E, off, w13, w2, act_bits=8)
    x = torch.randn(T, H, generator=g, device="cuda").half().requires_grad_()
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int()
    w = torch.rand(T, k, generator=g, device="cuda").requires_grad_()
    out = ex(x, ids, w)
    dout = torch.randn(T, H, generator=g, device="cuda").half()
    out.backward(dout)
    v13, v2, v13t, v2t = four(w13), four(w2), four(w13, True), four(w2, True)
    want, dx, dw = torch.zeros(T, H).double(), torch.zeros(T, H).double(), torch.zeros(T, k).double()
    xd, wd, dd = x.detach().cpu(), w.detach().double().cpu(), dout.double().cpu()
    le = ids.cpu().long() - off
    for e in range(El):
        t, j = torch.nonzero(le == e, as_tuple=True)
        if len(t):
            y, held = gated(xd[t], e, v13, v2, I)
            y = y.half().double()
            want.index_add_(0, t, wd[t, j][:, None] * y)
            dw[t, j] = (dd[t] * y).sum(1)
            dx.index_add_(0, t, gated_back((wd[t, j][:, None] * dd[t]).half(), held, e, v13t, v2t, I))
    assert rel(out, want) < TOL and rel(x.grad, dx) < TOL and rel(w.grad, dw) < TOL
    assert ex.get_status() == (moe.MOE_OK, 0)
    # what 4 bits give is finite, too
    assert torch.isfinite(MXExperts.from_master(E, off, w13, w2, backward=False)(x.detach(), ids, w.detach())).all()
