"""Trains a router and a linear adapter around frozen MXFP4 experts: every step is dispatch,
quantise, grouped product, gate, quantise, grouped product, weighted combine and their
gradients.

    python examples/mxfp4_experts.py [--tokens 2048] [--hidden 1024] [--inter 512] [--experts 32]
                                     [--top-k 4] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_mixture_experts_gb300.experts import MXExperts  # noqa: E402


def train(tokens=2048, hidden=1024, inter=512, experts=32, top_k=4, steps=20, lr=0.02, seed=0,
          say=print):
    """Losses of `steps` steps towards the output of another router over the same experts."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ex = MXExperts.from_master(experts, 0, randn(experts, 2 * inter, hidden) * hidden ** -0.5,
                               randn(experts, hidden, inter) * inter ** -0.5)
    target_router = randn(experts, hidden) * hidden ** -0.5

    def layer(x, router, adapter):
        h = x + x @ adapter
        logits, ids = (h.float() @ router.t()).topk(top_k, dim=1)
        return ex(h.bfloat16(), ids.int(), torch.softmax(logits, 1))

    router = (target_router + 0.5 * hidden ** -0.5 * randn(experts, hidden)).requires_grad_()
    adapter = (0.3 * hidden ** -0.5 * randn(hidden, hidden)).requires_grad_()
    opt = torch.optim.Adam([router, adapter], lr=lr * hidden ** -0.5)
    x = randn(tokens, hidden)
    with torch.no_grad():
        target = layer(x, target_router, torch.zeros_like(adapter)).float()
    losses = []
    for step in range(steps):
        loss = (layer(x, router, adapter).float() - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if say and step % 5 == 0:
            say("step %3d  loss %.4f" % (step, losses[-1].item()))
    losses = torch.stack(losses).tolist()
    status, bits = ex.get_status()
    if status:
        raise RuntimeError("errors found on the device: bits %#x" % bits)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 2048), ("hidden", 1024), ("inter", 512), ("experts", 32),
                          ("top-k", 4), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    out = train(a.tokens, a.hidden, a.inter, a.experts, a.top_k, a.steps)
    print("loss %.4f -> %.4f" % (out[0], out[-1]))
