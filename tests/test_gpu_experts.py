"""MXExperts (dispatch, quantise, product, gate, combine and their gradients together) against
the same layer written in 64 bits on the dequantised operands, and the example that trains
around it."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
import ops_ref as ref
from nvfp4_mixture_experts_gb300.experts import MXExperts, quantise

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def values(x, transpose=False, ceil=True):
    """fp64 of what x's MXFP4 form (of each matrix's transpose, with transpose) stands for."""
    m = x.detach().double().cpu().numpy()
    m = m[None] if m.ndim == 2 else m
    out = np.stack([ref.quant_mxfp4(a.T if transpose else a, ceil)[2] for a in m])
    return torch.from_numpy(out[0] if x.dim() == 2 else out)


def rel(a, b):
    return float((a.double().cpu() - b).norm() / b.norm())


@pytest.mark.parametrize("T,H,I,E,k,off,El", [(1, 64, 32, 4, 2, 0, 4), (37, 96, 64, 8, 3, 2, 5),
                                              (300, 160, 96, 6, 2, 0, 6)])
def test_layer_and_its_gradients(T, H, I, E, k, off, El):
    torch.manual_seed(T)
    w13 = torch.randn(El, 2 * I, H, device="cuda") * H ** -0.5
    w2 = torch.randn(El, H, I, device="cuda") * I ** -0.5
    ex = MXExperts.from_master(E, off, w13, w2)
    x = torch.randn(T, H, device="cuda", requires_grad=True)
    ids = torch.rand(T, E, device="cuda").topk(k, 1).indices.int()
    w = torch.rand(T, k, device="cuda", requires_grad=True)
    out = ex(x, ids, w)
    dout = torch.randn(T, H, device="cuda")
    out.backward(dout)

    # the layer pair by pair in 64 bits, on the operands' quantised values; activations and
    # gradients are quantised with the reference quantiser where the layer quantises them
    v13, v2, v13t, v2t = values(w13), values(w2), values(w13, True), values(w2, True)
    xq = values(x)
    want, dx, dw = torch.zeros(T, H).double(), torch.zeros(T, H).double(), torch.zeros(T, k).double()
    wd, dd = w.detach().double().cpu(), dout.double().cpu()
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j]) - off
            if not 0 <= e < El:
                continue
            gu = v13[e] @ xq[t]
            g, u = gu[:I], gu[I:]
            s = torch.sigmoid(g)
            act = (g * s * u).float()       # fp32 where the layer holds it in fp32
            y = v2[e] @ values(act[None])[0]
            want[t] += wd[t, j] * y
            dw[t, j] = dd[t] @ y
            ds = v2t[e] @ values((wd[t, j] * dd[t]).float()[None])[0]
            dgu = torch.cat((ds * u * s * (1 + g * (1 - s)), ds * g * s)).float()
            dx[t] += v13t[e] @ values(dgu[None])[0]
    # An fp32 value that lies within rounding of an E2M1 midpoint may round the other way and
    # moves its element by up to a third; with a share of 1e-3 of the elements doing so (the
    # midpoints' fp32 neighbourhoods are far rarer) the norms agree to 1e-2.
    assert rel(out.detach(), want) < 1e-2
    assert rel(x.grad, dx) < 1e-2
    assert rel(w.grad, dw) < 1e-2
    dropped = ((ids < off) | (ids >= off + El)).cpu()
    assert torch.all(w.grad.cpu()[dropped] == 0)


def test_checkpoint_form_gives_the_same_layer():
    torch.manual_seed(3)
    E, H, I, T, k = 5, 160, 64, 40, 2
    w13 = torch.randn(E, 2 * I, H, device="cuda")
    w2 = torch.randn(E, H, I, device="cuda")
    parts = []
    for m in (w13, w2):
        rows, cols = m.shape[1:]
        codes = torch.empty(E, rows, cols // 2, dtype=torch.uint8, device="cuda")
        sf = torch.empty(E, rows, cols // 32, dtype=torch.uint8, device="cuda")
        moe.moe_quant_mxfp4(m, codes, sf, moe.MOE_SF_CANONICAL, scale_rule=moe.MOE_MX_CEIL)
        parts += [codes, sf]
    x = torch.randn(T, H, device="cuda").bfloat16()
    ids = torch.rand(T, E, device="cuda").topk(k, 1).indices.int()
    w = torch.rand(T, k, device="cuda")
    a = MXExperts.from_checkpoint(E, 0, *parts)(x, ids, w)
    b = MXExperts.from_master(E, 0, w13, w2, backward=False)(x, ids, w)
    assert torch.equal(a, b)
    x.requires_grad_()
    with pytest.raises(RuntimeError):
        MXExperts.from_checkpoint(E, 0, *parts)(x, ids, w).sum().backward()


def test_shards_add_up():
    torch.manual_seed(4)
    E, H, I, T, k = 6, 128, 64, 50, 3
    w13, w2 = torch.randn(E, 2 * I, H, device="cuda"), torch.randn(E, H, I, device="cuda")
    x = torch.randn(T, H, device="cuda")
    ids = torch.rand(T, E, device="cuda").topk(k, 1).indices.int()
    w = torch.rand(T, k, device="cuda")

    def shard(lo, hi):
        ex = MXExperts.from_master(E, lo, w13[lo:hi], w2[lo:hi], backward=False)
        return ex(x, ids, w).double()

    one = [shard(e, e + 1) for e in range(E)]     # single terms w y, rounded once
    mag = sum(o.abs() for o in one)
    # k terms in fp32 in any grouping: k roundings of at most the magnitudes' sum
    for parts in ([shard(0, E)], [shard(0, 2), shard(2, E)]):
        assert torch.all((sum(parts) - sum(one)).abs() <= (k + 1) * 2.0 ** -23 * mag)


def test_no_tokens():
    ex = MXExperts.from_master(4, 0, torch.randn(4, 64, 32, device="cuda"), torch.randn(4, 32, 32, device="cuda"))
    x = torch.zeros(0, 32, device="cuda", requires_grad=True)
    w = torch.zeros(0, 2, device="cuda", requires_grad=True)
    out = ex(x, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), w)
    out.sum().backward()
    assert out.shape == (0, 32) and x.grad.shape == (0, 32) and w.grad.shape == (0, 2)


def test_quantise_pads_nothing():
    x = torch.randn(3, 64, device="cuda")
    codes, sf = quantise(x)
    assert codes.shape == (3, 32) and sf.numel() == 512
    codes, sf = quantise(torch.randn(2, 32, 5, device="cuda"), transpose=True)
    assert codes.shape == (2, 5, 16) and sf.numel() == 2 * 512


def test_example_trains():
    spec = importlib.util.spec_from_file_location(
        "mxfp4_experts_example", os.path.join(ROOT, "examples", "mxfp4_experts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.train(tokens=512, hidden=256, inter=128, experts=8, top_k=2, steps=30, say=None)
    assert all(np.isfinite(losses)) and losses[-1] < 0.7 * losses[0]
