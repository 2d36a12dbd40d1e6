"""MXBlock: the mixture-of-experts half of a transformer block around frozen MXFP4 experts, forward and
backward -- the norm with the residual's addition, routing, the experts and the shared expert.

rms_norm and route are the block's own operators for autograd; their gradients, like the experts',
have none of their own (second derivatives raise).  A step with its backward pass can be captured into a
CUDA graph, as with torch's own operators once nothing holds an eager step's results: autograd ties the
leaves' gradients to the stream of the oldest graph of theirs that is alive, which must not be another one.
"""
import torch

from . import (MOE_GROUP_MAX, MOE_SCORE_SOFTMAX, MOE_SF_TILED, moe_mxfp4_scale_bytes, moe_rmsnorm,
               moe_rmsnorm_backward, moe_rmsnorm_workspace_size, moe_route_scores,
               moe_route_scores_backward)
from .experts import _FirstOrder, as_rows


def rms_norm(x, weight, eps=1e-6, residual=None, eight=False):
    """(y, h, codes, scales) for rows x [T, H]: h = x + residual (x where there is none), y = h /
    sqrt(mean h^2 + eps) * weight, and with eight y's MXFP8 matrix with tiled scales (None without; it
    has no gradient of its own: what reads it passes its gradient to y).  Differentiable in x, residual
    and weight, through y and h.  The weight may be of any float type; it is rounded to x's for the product,
    and its gradient to the weight's."""
    y, h, codes, sf = _Norm.apply(x, residual, weight, eps, eight)
    return y, x if residual is None else h, codes, sf


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, eight):
        T, H = x.shape
        x = as_rows(x)
        y = torch.empty(T, H, dtype=x.dtype, device=x.device)
        rstd = torch.empty(T, dtype=torch.float32, device=x.device)
        w = weight.detach().to(x.dtype).contiguous()
        h = codes = sf = None
        if residual is not None:
            residual = as_rows(residual)
            h = torch.empty_like(y)
        if eight:
            codes = torch.empty(T, H, dtype=torch.uint8, device=x.device)
            sf = torch.empty(moe_mxfp4_scale_bytes(1, T, H, MOE_SF_TILED), dtype=torch.uint8, device=x.device)
        moe_rmsnorm(x, w, eps, residual=residual, h=h, y=y, rstd=rstd, codes=codes, sf=sf)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x if h is None else h, w, rstd)
        ctx.weight_dtype = weight.dtype
        if eight:
            ctx.mark_non_differentiable(codes, sf)
        return y, h, codes, sf

    @staticmethod
    def backward(ctx, dy, dh, *_):
        with torch.no_grad():
            dx, dw = _Norm.gradients(ctx, dy, dh)
        if torch.is_grad_enabled():
            dx, dw = _FirstOrder.apply("rms_norm", dx.requires_grad_(), dw.requires_grad_())
        need = ctx.needs_input_grad
        return dx, dx if need[1] else None, dw if need[2] else None, None, None

    @staticmethod
    def gradients(ctx, dy, dh):
        h, w, rstd = ctx.saved_tensors
        T, H = h.shape
        if dy is None:   # y is not used: its gradient is zero
            dy = torch.zeros(T, H, dtype=h.dtype, device=h.device)
        dx, dw = torch.empty(T, H, dtype=h.dtype, device=h.device), None
        ws = None
        if ctx.needs_input_grad[2]:
            dw = torch.empty(H, dtype=torch.float32, device=h.device)
            ws = torch.empty(moe_rmsnorm_workspace_size(T, H), dtype=torch.uint8, device=h.device)
        moe_rmsnorm_backward(as_rows(dy), h, w, rstd, dx, dw, ws,
                             dh=None if dh is None else as_rows(dh))
        return dx, torch.zeros(H, dtype=ctx.weight_dtype, device=h.device) if dw is None else dw.to(ctx.weight_dtype)


def route(logits, k, bias=None, score=MOE_SCORE_SOFTMAX, num_groups=1, topk_groups=1,
          group_score=MOE_GROUP_MAX, renormalise=True, scale=1.0):
    """(ids int32 [T, k], weights float32 [T, k]) of moe_route_scores; the weights are differentiable in
    the logits."""
    return _Route.apply(logits, k, bias, score, num_groups, topk_groups, group_score, renormalise, scale)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, bias, score, num_groups, topk_groups, group_score, renormalise, scale):
        T = logits.shape[0]
        logits = as_rows(logits)
        ids = torch.empty(T, k, dtype=torch.int32, device=logits.device)
        w = torch.empty(T, k, dtype=torch.float32, device=logits.device)
        moe_route_scores(logits, ids, w, bias=bias, score=score, num_groups=num_groups,
                         topk_groups=topk_groups, group_score=group_score, renormalise=renormalise, scale=scale)
        ctx.save_for_backward(logits, ids)
        ctx.how = dict(score=score, renormalise=renormalise, scale=scale)
        ctx.mark_non_differentiable(ids)
        return ids, w

    @staticmethod
    def backward(ctx, _, dw):
        logits, ids = ctx.saved_tensors
        with torch.no_grad():
            d = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
            moe_route_scores_backward(logits, ids, dw.float().contiguous(), d, **ctx.how)
        if torch.is_grad_enabled():
            d, = _FirstOrder.apply("route", d.requires_grad_())
        return (d,) + (None,) * 8


class MXBlock:
    """h = x + residual; y = rms_norm(h); out = experts(y, route(y router^T)) [+ shared(y)].

    norm_weight [H] and router [num_experts, H] are the caller's leaves, of any float type: the norm's weight is
    rounded to x's on every call, y to the router's for the logits, which are torch's matrix product in that
    type.  experts: an MXExperts (of a shard: out is its partial sum); shared: an MXShared (of several shards
    one has it) or None; the other arguments are route's."""

    def __init__(self, norm_weight, router, experts, top_k, shared=None, eps=1e-6, **routing):
        self.norm_weight, self.router, self.experts, self.shared = norm_weight, router, experts, shared
        self.top_k, self.eps, self.routing = top_k, eps, routing

    def __call__(self, x, residual=None):
        """(out, h), both [T, H] in x's type: the next block's x and residual."""
        y, h, codes, sf = rms_norm(x, self.norm_weight, self.eps, residual, eight=self.shared is not None)
        logits = y.to(self.router.dtype) @ self.router.t()
        ids, w = route(logits, self.top_k, **self.routing)
        out = self.experts(y, ids, w)
        if self.shared is not None:
            out = out + self.shared(y, (codes, sf))
        return out, h

    def get_status(self):
        """(status, bits) of the experts (MXExperts.get_status), or of the shared expert where those have
        found nothing."""
        status, bits = self.experts.get_status()
        if status or self.shared is None:
            return status, bits
        return self.shared.get_status()
