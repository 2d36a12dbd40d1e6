"""What the experts' buffers hold before a call does not reach its results: every floating-point and byte buffer
that the layers make is filled first, with zeros or with ones in all bits (NaN, as codes and as scales too)."""
import types

import pytest
import torch

from nvfp4_mixture_experts_gb300 import block, experts
from nvfp4_mixture_experts_gb300.experts import MXExperts, MXShared
from test_gpu_block import masters

pytestmark = pytest.mark.gpu


class Filled(types.ModuleType):
    """torch, but for empty and empty_like, whose tensors hold `byte` in every byte (integers of 32 bits, which
    are maps that the library bounds, are left alone)."""

    def __init__(self, byte):
        super().__init__("torch")
        self.byte, self.made = byte, []

    def __getattr__(self, name):
        return getattr(torch, name)

    def fill(self, t):
        if t.dtype != torch.int32:
            t.view(-1).view(torch.uint8).fill_(self.byte)
            self.made.append(t.numel())
        return t

    def empty(self, *a, **kw):
        return self.fill(torch.empty(*a, **kw))

    def empty_like(self, t):
        return self.fill(torch.empty(t.shape, dtype=t.dtype, device=t.device))


def both(monkeypatch, f):
    results = []
    for byte in (0, 255):
        t = Filled(byte)
        monkeypatch.setattr(experts, "torch", t)
        monkeypatch.setattr(block, "torch", t)
        results.append(f())
        assert len(t.made) >= 5
    for a, b in zip(*results):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


@pytest.mark.parametrize("act_bits", [4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_experts(monkeypatch, act_bits, dtype):
    g = torch.Generator("cuda").manual_seed(0)
    w13, w2 = masters(5, 256, 128, g)
    ex = MXExperts.from_master(9, 2, w13, w2, act_bits=act_bits)
    x = torch.randn(60, 256, generator=g, device="cuda").to(dtype)
    ids = torch.rand(60, 9, generator=g, device="cuda").topk(2, 1).indices.int()
    ids[ids == 4] = 8          # an expert with no rows
    w = torch.rand(60, 2, generator=g, device="cuda")
    dout = torch.randn(60, 256, generator=g, device="cuda").to(dtype)

    def step():
        a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
        y = ex(a, ids, b)
        y.backward(dout)
        return y.detach(), a.grad, b.grad

    both(monkeypatch, step)


@pytest.mark.parametrize("T", [1, 60, 300])
def test_shared_expert_and_block(monkeypatch, T):
    g = torch.Generator("cuda").manual_seed(T)
    w13, w2 = masters(6, 128, 128, g)
    s13, s2 = masters(1, 128, 128, g)
    bl = block.MXBlock(torch.ones(128, device="cuda").requires_grad_(),
                       (torch.randn(6, 128, generator=g, device="cuda") * 0.1).requires_grad_(),
                       MXExperts.from_master(6, 0, w13, w2, act_bits=8), 2, shared=MXShared.from_master(s13, s2))
    x, r, dout = (torch.randn(T, 128, generator=g, device="cuda").bfloat16() for _ in range(3))

    def step():
        a, b = x.clone().requires_grad_(), r.clone().requires_grad_()
        out, h = bl(a, b)
        grads = torch.autograd.grad((out, h), (a, b, bl.norm_weight, bl.router), (dout, dout))
        shared = bl.shared(a)
        return (out.detach(), h.detach(), shared.detach(), *grads, *torch.autograd.grad(shared, (a,), (dout,)))

    both(monkeypatch, step)
