"""The operators around the experts used together: MXExperts and MXShared with 8-bit activations, and
MXBlock (norm, routing, experts, shared expert) with its gradients, against the same layers written in 64
bits on the quantised operands."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
import ops8_ref as ref
import ops_ref
from nvfp4_mixture_experts_gb300.block import MXBlock, rms_norm, route
from nvfp4_mixture_experts_gb300.experts import MXExperts, MXShared, quantise8

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def four(x, transpose=False):
    """fp64 of what x's MXFP4 form (of each matrix's transpose) stands for."""
    m = x.detach().double().cpu().numpy()
    return torch.from_numpy(np.stack([ops_ref.quant_mxfp4(a.T if transpose else a, True)[2] for a in m]))


def eight(x):
    """fp64 of what the rows' MXFP8 form stands for."""
    return torch.from_numpy(ref.quant_mxfp8(x.double().numpy(), True)[2])


def gated(x, e, v13, v2, I, hold=torch.float32):
    """(down rows, what the backward pass needs) of rows x through expert e; hold: the type that the
    products' results are held in."""
    gu = (eight(x) @ v13[e].T).to(hold).double()
    held = eight(gu.float())
    return eight((torch.from_numpy(ref.swiglu(gu[:, :I].numpy(), gu[:, I:].numpy()))).float()) @ v2[e].T, held


def gated_back(dy, held, e, v13t, v2t, I, hold=torch.float32):
    ds = (eight(dy.float()) @ v2t[e].T).to(hold).double()
    dg, du = ref.swiglu_grad(ds.numpy(), held[:, :I].numpy(), held[:, I:].numpy())
    return eight(torch.from_numpy(np.concatenate([dg, du], 1)).float()) @ v13t[e].T


def rel(a, b):
    return float((a.detach().double().cpu() - b).norm() / b.norm())


# An fp32 value within rounding of a midpoint of two E4M3 numbers may round the other way and move its
# element by an eighth: with a share of 1e-4 of the elements doing so (fp32 neighbourhoods are far rarer)
# the norms agree to 1/8 of its root, 1.3e-3, in each of at most six roundings on a path.
TOL = 1e-2


def masters(E, H, I, g):
    w13 = torch.randn(E, 2 * I, H, generator=g, device="cuda") * H ** -0.5
    return w13, torch.randn(E, H, I, generator=g, device="cuda") * I ** -0.5


@pytest.mark.parametrize("T,H,I,E,k,off,El", [(1, 128, 128, 4, 2, 0, 4), (37, 256, 128, 8, 3, 2, 5),
                                              (300, 128, 384, 6, 2, 0, 6)])
def test_experts_and_their_gradients(T, H, I, E, k, off, El):
    g = torch.Generator("cuda").manual_seed(T)
    w13, w2 = masters(El, H, I, g)
    ex = MXExperts.from_master(E, off, w13, w2, act_bits=8)
    x = torch.randn(T, H, generator=g, device="cuda", requires_grad=True)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int()
    w = torch.rand(T, k, generator=g, device="cuda").requires_grad_()
    out = ex(x, ids, w)
    dout = torch.randn(T, H, generator=g, device="cuda")
    out.backward(dout)
    v13, v2, v13t, v2t = four(w13), four(w2), four(w13, True), four(w2, True)
    want, dx, dw = torch.zeros(T, H).double(), torch.zeros(T, H).double(), torch.zeros(T, k).double()
    xd, wd, dd = x.detach().cpu(), w.detach().double().cpu(), dout.double().cpu()
    le = ids.cpu().long() - off
    for e in range(El):
        t, j = torch.nonzero(le == e, as_tuple=True)
        if len(t):
            y, held = gated(xd[t], e, v13, v2, I)
            y = y.float().double()
            want.index_add_(0, t, wd[t, j][:, None] * y)
            dw[t, j] = (dd[t] * y).sum(1)
            dx.index_add_(0, t, gated_back(wd[t, j][:, None] * dd[t], held, e, v13t, v2t, I))
    assert rel(out, want) < TOL and rel(x.grad, dx) < TOL and rel(w.grad, dw) < TOL
    assert torch.all(w.grad.cpu()[(le < 0) | (le >= El)] == 0)
    assert ex.get_status() == (moe.MOE_OK, 0)
    # 8 bits are nearer to the unquantised activations than 4
    plain = torch.zeros(T, H).double()
    for e in range(El):
        t, j = torch.nonzero(le == e, as_tuple=True)
        gu = xd[t].double() @ v13[e].T
        plain.index_add_(0, t, wd[t, j][:, None] * (torch.from_numpy(ref.swiglu(gu[:, :I].numpy(), gu[:, I:].numpy())) @ v2[e].T))
    if T > 1:
        in4 = MXExperts.from_master(E, off, w13, w2, backward=False)(x.detach(), ids, w.detach())
        assert rel(out, plain) < 0.5 * rel(in4, plain)


@pytest.mark.parametrize("T,H,I", [(1, 128, 128), (150, 256, 384)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shared_expert(T, H, I, dtype):
    g = torch.Generator("cuda").manual_seed(I)
    w13, w2 = masters(1, H, I, g)
    sh = MXShared.from_master(w13, w2)
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype).requires_grad_()
    out = sh(x)
    dout = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    out.backward(dout)
    y, held = gated(x.detach().cpu(), 0, four(w13), four(w2), I, dtype)
    dx = gated_back(dout.cpu(), held, 0, four(w13, True), four(w2, True), I, dtype)
    assert rel(out, y) < TOL and rel(x.grad, dx) < TOL
    assert torch.equal(out, sh(x, quantise8(x.detach())))
    assert sh.get_status() == (moe.MOE_OK, 0)


def test_weights_of_a_checkpoint():
    """The same codes with canonical scales."""
    g = torch.Generator("cuda").manual_seed(2)
    H, I = 128, 256
    w13, w2 = masters(3, H, I, g)
    kept = []
    for w in (w13, w2):
        codes = torch.empty(*w.shape[:2], w.shape[2] // 2, dtype=torch.uint8, device="cuda")
        sf = torch.empty(*w.shape[:2], w.shape[2] // 32, dtype=torch.uint8, device="cuda")
        moe.moe_quant_mxfp4(w, codes, sf, moe.MOE_SF_CANONICAL, scale_rule=moe.MOE_MX_CEIL)
        kept += [codes, sf]
    x = torch.randn(50, H, generator=g, device="cuda").bfloat16()
    ids = torch.rand(50, 3, generator=g, device="cuda").topk(2, 1).indices.int()
    w = torch.rand(50, 2, generator=g, device="cuda")
    a = MXExperts.from_checkpoint(3, 0, *kept, act_bits=8)(x, ids, w)
    assert torch.equal(a, MXExperts.from_master(3, 0, w13, w2, backward=False, act_bits=8)(x, ids, w))
    b = MXShared.from_checkpoint(*(t[:1].contiguous() for t in kept))(x)
    assert torch.equal(b, MXShared.from_master(w13[:1], w2[:1], backward=False)(x))


def test_padding_rows_are_not_read_and_results_repeat():
    g = torch.Generator("cuda").manual_seed(0)
    w13, w2 = masters(5, 128, 128, g)
    ex = MXExperts.from_master(5, 0, w13, w2, act_bits=8)
    x = torch.randn(60, 128, generator=g, device="cuda").bfloat16()
    ids = torch.rand(60, 5, generator=g, device="cuda").topk(2, 1).indices.int()
    w = torch.rand(60, 2, generator=g, device="cuda")
    outs = []
    for fill in (0.0, float("nan")):
        junk = [torch.full((1 << 20,), fill, device="cuda") for _ in range(8)]   # what the buffers hold before
        del junk
        a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
        y = ex(a, ids, b)
        y.float().square().sum().backward()
        outs.append((y.detach(), a.grad, b.grad))
    assert all(torch.equal(p, q) for p, q in zip(*outs))
    assert all(torch.isfinite(t.float()).all() for t in outs[0])


def block(T, H, I, E, k, g, shared=True, **kw):
    w13, w2 = masters(E, H, I, g)
    s13, s2 = masters(1, H, I, g)
    ex = MXExperts.from_master(E, 0, w13, w2, act_bits=8)
    sh = MXShared.from_master(s13, s2) if shared else None
    norm = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).requires_grad_()
    router = (torch.randn(E, H, generator=g, device="cuda") * H ** -0.5).requires_grad_()
    return MXBlock(norm, router, ex, k, shared=sh, **kw), (w13, w2, s13, s2)


@pytest.mark.parametrize("kind,groups,renorm", [("softmax", 1, True), ("sigmoid", 4, True), ("softmax", 2, False)])
def test_block_and_its_gradients(kind, groups, renorm):
    T, H, I, E, k, eps = 90, 256, 128, 8, 2, 1e-5
    g = torch.Generator("cuda").manual_seed(groups)
    bias = torch.randn(E, generator=g, device="cuda") * 0.05
    score = moe.MOE_SCORE_SOFTMAX if kind == "softmax" else moe.MOE_SCORE_SIGMOID
    bl, (w13, w2, s13, s2) = block(T, H, I, E, k, g, eps=eps, bias=bias, score=score, num_groups=groups,
                                   topk_groups=max(1, groups // 2), renormalise=renorm, scale=2.0)
    x, r = (torch.randn(T, H, generator=g, device="cuda").requires_grad_() for _ in range(2))
    out, h = bl(x, r)
    dout, dh = (torch.randn(T, H, generator=g, device="cuda") for _ in range(2))
    torch.autograd.backward((out, h), (dout, dh))
    assert bl.get_status() == (moe.MOE_OK, 0)

    # in 64 bits, by hand
    h64 = (x + r).detach().double().cpu().numpy()
    wn, wr = bl.norm_weight.detach().double().cpu().numpy(), bl.router.detach().double().cpu().numpy()
    y, rstd = ref.rmsnorm(h64, wn, eps)
    logits = y @ wr.T
    ids, w = ref.route(logits, bias.double().cpu().numpy(), k, kind, groups, max(1, groups // 2), False, renorm, 2.0)
    v = [four(m) for m in (w13, w2, s13, s2)]
    vt = [four(m, True) for m in (w13, w2, s13, s2)]
    yt, dd = torch.from_numpy(y).float(), dout.double().cpu()
    want, held_s = gated(yt, 0, v[2], v[3], I)
    dy = gated_back(dout.cpu(), held_s, 0, vt[2], vt[3], I).numpy()
    dw = np.zeros((T, k))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if len(t):
            rows, held = gated(yt[t], e, v[0], v[1], I)
            wt = torch.from_numpy(w[t, j])[:, None]
            want.index_add_(0, torch.from_numpy(t), wt * rows)
            dw[t, j] = (dd[t] * rows).sum(1)
            np.add.at(dy, t, gated_back(wt * dd[t], held, e, vt[0], vt[1], I).numpy())
    dl = ref.route_grad(logits, ids, dw, kind, renorm, 2.0)
    dy += dl @ wr
    dx, dwn = ref.rmsnorm_grad(dy, h64, wn, rstd, dh.double().cpu().numpy())
    as_t = torch.from_numpy
    assert rel(h, as_t(h64)) < 1e-6
    assert rel(out, want) < TOL
    assert rel(x.grad, as_t(dx)) < TOL and torch.equal(x.grad, r.grad)
    assert rel(bl.norm_weight.grad, as_t(dwn)) < TOL and rel(bl.router.grad, as_t(dl.T @ y)) < TOL


def test_block_in_16_bits_chained_without_residual():
    g = torch.Generator("cuda").manual_seed(3)
    a, _ = block(40, 128, 128, 4, 2, g)
    b, _ = block(40, 128, 128, 4, 2, g, shared=False)
    x = torch.randn(40, 128, generator=g, device="cuda").bfloat16().requires_grad_()
    out, h = a(x)
    assert h is x
    out, h = b(out, h)
    (out + h).float().square().mean().backward()
    for t in (x, a.norm_weight, a.router, b.norm_weight, b.router):
        assert t.grad is not None and t.grad.shape == t.shape and t.grad.dtype == t.dtype
        assert torch.isfinite(t.grad.float()).all() and bool((t.grad != 0).any())


def test_block_of_no_tokens():
    g = torch.Generator("cuda").manual_seed(4)
    bl, _ = block(0, 128, 128, 4, 2, g)
    x = torch.empty(0, 128, device="cuda", requires_grad=True)
    out, h = bl(x, torch.empty(0, 128, device="cuda"))
    (out.sum() + h.sum()).backward()
    assert out.shape == (0, 128) and x.grad.shape == (0, 128) and torch.all(bl.norm_weight.grad == 0)


def test_norm_alone():
    x = torch.randn(5, 64, device="cuda", requires_grad=True)
    r = torch.randn(5, 64, device="cuda")
    w = torch.rand(64, device="cuda")
    y, h, codes, sf = rms_norm(x, w, residual=r)
    assert codes is None and sf is None
    h.sum().backward()                       # y unused
    assert torch.equal(x.grad, torch.ones_like(x))
    y, h, codes, sf = rms_norm(x.detach()[:, :32].double().float(), w[:32], eight=True)
    assert codes.shape == (5, 32) and not y.requires_grad
    x.grad = None
    y, _, _, _ = rms_norm(x, w.requires_grad_(), residual=r)
    dx, dw = torch.autograd.grad(y.square().sum(), (x, w), create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        (dx.sum() + dw.sum()).backward()


def test_rows_that_repeat_or_are_transposed():
    """Inputs and gradients that are broadcast over the tokens or transposed: the results of their copies."""
    g = torch.Generator("cuda").manual_seed(5)
    T, H = 9, 128
    w13, w2 = masters(1, H, H, g)
    sh = MXShared.from_master(w13, w2)
    one, wide = torch.randn(H, generator=g, device="cuda"), torch.randn(H, T, generator=g, device="cuda")
    r = torch.randn(1, H, generator=g, device="cuda", requires_grad=True)
    v = torch.randn(2, H, generator=g, device="cuda")
    w = torch.rand(H, generator=g, device="cuda")
    for x in (one.expand(T, H), wide.t()):
        results = []
        for copy in (False, True):
            r.grad = None
            a = (x.clone(memory_format=torch.contiguous_format) if copy else x.detach()).requires_grad_()
            res = r.expand(T, H)
            y, h, _, _ = rms_norm(a, w, residual=res.contiguous() if copy else res)
            vy, vh = (u.expand(T, H).contiguous() if copy else u.expand(T, H) for u in v)
            da, dr = torch.autograd.grad((y, h), (a, r), (vy, vh), retain_graph=True)
            results.append((y, h, da, dr, *route(a, 4), sh(a)))
        assert all(torch.equal(p, q) for p, q in zip(*results))


def test_route_second_derivatives_raise():
    l = torch.randn(3, 8, device="cuda", requires_grad=True)
    _, w = route(l, 2)
    d, = torch.autograd.grad(w.square().sum(), l, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        d.sum().backward()


def test_block_in_a_graph():
    """Forward and backward of the block captured and replayed on other inputs."""
    g = torch.Generator("cuda").manual_seed(6)
    bl, _ = block(64, 256, 128, 8, 2, g)
    x = torch.randn(64, 256, generator=g, device="cuda").bfloat16().requires_grad_()
    r = torch.randn(64, 256, generator=g, device="cuda").bfloat16().requires_grad_()
    leaves = (x, r, bl.norm_weight, bl.router)

    def step():
        out, h = bl(x, r)
        return (out.detach(), *torch.autograd.grad((out.float().square().sum() + h.float().sum()), leaves))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        x.copy_(torch.randn(64, 256, generator=g, device="cuda"))
        r.copy_(torch.randn(64, 256, generator=g, device="cuda"))
    graph.replay()
    kept = [t.clone() for t in got]
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))


def test_example_runs_with_8_bit_activations():
    spec = importlib.util.spec_from_file_location(
        "mxfp4_experts_example", os.path.join(ROOT, "examples", "mxfp4_experts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.train(tokens=256, hidden=256, inter=128, experts=8, top_k=2, steps=3, say=None, act_bits=8)
    assert len(losses) == 3 and all(np.isfinite(losses))
