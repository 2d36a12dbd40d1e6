"""MXExperts: a shard of gated experts with frozen MXFP4 weights, forward and backward.

The handle-free operators in the order a training step (or a forward that wants gradients later)
calls them:

  forward   moe_dispatch -> moe_quant_mxfp4 -> moe_grouped_gemm_mxfp4 (gate_up) -> silu(g) * u
            -> moe_quant_mxfp4 -> moe_grouped_gemm_mxfp4 (down) -> moe_combine_weighted
  backward  moe_combine_backward -> moe_quant_mxfp4 -> product with W2^T -> the gate's gradient
            -> moe_quant_mxfp4 -> product with W13^T -> moe_dispatch_backward

The quantisation of activations and gradients is passed straight through; the weights (adapters
and routers train around them) have no gradient, and the gradients have none (second derivatives
raise).  The elementwise gate is torch's, on all rows of
the sorted buffers: rows of no pair hold stale values that nothing downstream reads.
"""
import torch

from . import (MOE_DEV_WAIT_TIMEOUT, MOE_ERR_DEVICE_STATUS, MOE_ERR_TIMEOUT, MOE_ERR_UNSUPPORTED,
               MOE_MX_CEIL, MOE_OK, MOE_SF_TILED, MoEError, moe_combine_backward,
               moe_combine_weighted, moe_dispatch, moe_dispatch_backward,
               moe_dispatch_rows_capacity, moe_grouped_gemm_mxfp4, moe_mxfp4_scale_bytes,
               moe_mxfp4_tile_scales, moe_quant_mxfp4)

ROW_ALIGN = 128  # groups start on whole row blocks of scales, as the product reads them


def quantise(x, transpose=False, perm_src=None, scale_rule=MOE_MX_CEIL):
    """(codes, tiled scales) of x [rows, cols] or [batch, rows, cols], or of its transpose."""
    rows, cols = x.shape[-2:][::-1] if transpose else x.shape[-2:]
    batch = x.shape[0] if x.dim() == 3 else 1
    codes = torch.empty((*x.shape[:-2], rows, cols // 2), dtype=torch.uint8, device=x.device)
    sf = torch.empty(moe_mxfp4_scale_bytes(batch, rows, cols, MOE_SF_TILED), dtype=torch.uint8,
                     device=x.device)
    moe_quant_mxfp4(x, codes, sf, MOE_SF_TILED, transpose=transpose, scale_rule=scale_rule,
                    perm_src=perm_src)
    return codes, sf


class MXExperts:
    """Experts local_off .. local_off + num_local - 1 of num_experts: w13 [num_local, 2I, H] (gate
    rows, then up rows) and w2 [num_local, H, I], H and I multiples of 32."""

    def __init__(self, num_experts, local_off, w13, w13_sf, w2, w2_sf, w13_t=None, w2_t=None):
        """w13, w2: MXFP4 codes [num_local, rows, cols / 2] with tiled scales w13_sf, w2_sf.  w13_t,
        w2_t: (codes, scales) of each expert's transposed matrices; without them there is no
        backward."""
        self.num_experts, self.local_off = num_experts, local_off
        self.num_local, two_inter, half_hidden = w13.shape
        self.hidden, self.inter = 2 * half_hidden, two_inter // 2
        self.w13, self.w2, self.w13_t, self.w2_t = (w13, w13_sf), (w2, w2_sf), w13_t, w2_t
        self.status = torch.zeros(1, dtype=torch.int32, device=w13.device)

    @classmethod
    def from_master(cls, num_experts, local_off, w13, w2, backward=True):
        """Quantises bf16/fp16/fp32 master weights; for the backward pass their transposes too
        (blocks of 32 run along the contraction, so a transpose has its own codes)."""
        return cls(num_experts, local_off, *quantise(w13), *quantise(w2),
                   quantise(w13, transpose=True) if backward else None,
                   quantise(w2, transpose=True) if backward else None)

    @classmethod
    def from_checkpoint(cls, num_experts, local_off, w13, w13_sf, w2, w2_sf):
        """Codes and canonical scales [num_local, rows, cols / 32] of a checkpoint (forward only)."""
        tiled = []
        for codes, sf in ((w13, w13_sf), (w2, w2_sf)):
            n, rows, cols = codes.shape[0], codes.shape[1], codes.shape[2] * 2
            t = torch.empty(moe_mxfp4_scale_bytes(n, rows, cols, MOE_SF_TILED), dtype=torch.uint8,
                            device=codes.device)
            moe_mxfp4_tile_scales(sf, n, rows, cols, t)
            tiled += [codes, t]
        return cls(num_experts, local_off, *tiled)

    def __call__(self, x, topk_ids, topk_w):
        """The shard's partial sum [T, H] in x's type for tokens x [T, H] routed to topk_ids
        (int32 [T, k]) with weights topk_w (float32 [T, k]); differentiable in x and topk_w.
        Asynchronous: errors found on the device are read with get_status."""
        return _Experts.apply(x, topk_w, topk_ids, self)


    def get_status(self):
        """(status, bits), as moe_get_status: waits for the current stream, reads the MOE_DEV_* bits
        that the forwards and backwards since the last reading found on the device (an expert id out
        of range, whose pair was dropped; a wait that ran out, whose results are incomplete) and
        clears them.  MOE_OK, MOE_ERR_TIMEOUT or MOE_ERR_DEVICE_STATUS."""
        bits = self.status.item()
        self.status.zero_()
        if bits & MOE_DEV_WAIT_TIMEOUT:
            return MOE_ERR_TIMEOUT, bits
        return (MOE_ERR_DEVICE_STATUS if bits else MOE_OK), bits


class _FirstOrder(torch.autograd.Function):
    """Gradients that are part of a graph (create_graph) and have no gradient of their own."""

    @staticmethod
    def forward(ctx, *grads):
        return tuple(g.clone() for g in grads)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("MXExperts has no second derivatives")


class _Experts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, topk_w, topk_ids, ex):
        (T, k), dev, dt = topk_ids.shape, x.device, x.dtype
        cap = moe_dispatch_rows_capacity(T, k, ex.num_local, ROW_ALIGN)
        if T and not cap:  # rows of no capacity would hold no pair
            raise MoEError(MOE_ERR_UNSUPPORTED, "MXExperts: %d tokens, top-%d" % (T, k))
        i32 = dict(dtype=torch.int32, device=dev)
        counts, offsets = torch.empty(ex.num_local, **i32), torch.empty(ex.num_local + 1, **i32)
        perm, inv = torch.empty(cap, **i32), torch.empty(T * k, **i32)
        rows = torch.empty(cap, ex.hidden, dtype=dt, device=dev)
        moe_dispatch(x, topk_ids, ex.num_experts, ex.local_off, ex.num_local, ROW_ALIGN, counts,
                     offsets, perm, inv, rows, ex.status)

        def product(a, w, cols, dtype):
            out = torch.empty(cap, cols, dtype=dtype, device=dev)
            moe_grouped_gemm_mxfp4(*quantise(a, perm_src=perm), counts, offsets, *w, out,
                                   status=ex.status)
            return out

        gu = product(rows, ex.w13, 2 * ex.inter, torch.float32)
        gate, up = gu[:, :ex.inter], gu[:, ex.inter:]
        y = product(torch.nn.functional.silu(gate) * up, ex.w2, ex.hidden, dt)
        w = topk_w.detach().float().contiguous()
        out = torch.empty(T, ex.hidden, dtype=dt, device=dev)
        moe_combine_weighted(y, inv, w, out)
        ctx.ex, ctx.product, ctx.k = ex, product, k
        ctx.save_for_backward(gu, y, w, inv)
        return out

    @staticmethod
    def backward(ctx, dout):
        with torch.no_grad():
            grads = _Experts.gradients(ctx, dout)
        # Under create_graph the gradients depend on x, topk_w and dout, but the kernels leave no
        # graph: a second derivative must not be taken for zero.
        if torch.is_grad_enabled():
            grads = _FirstOrder.apply(*(g.requires_grad_() for g in grads))
        return (*grads, None, None)

    @staticmethod
    def gradients(ctx, dout):
        ex, k = ctx.ex, ctx.k
        if ex.w13_t is None:
            raise RuntimeError("MXExperts without transposed weights has no backward")
        gu, y, w, inv = ctx.saved_tensors
        dout = dout.to(y.dtype).contiguous()
        dy, dw = torch.empty_like(y), torch.empty_like(w)
        moe_combine_backward(dout, y, inv, w, dy, dw)
        ds = ctx.product(dy, ex.w2_t, ex.inter, torch.float32)
        gate, up = gu[:, :ex.inter], gu[:, ex.inter:]
        s = torch.sigmoid(gate)
        dgu = torch.cat((ds * up * s * (1 + gate * (1 - s)), ds * gate * s), 1)
        drows = ctx.product(dgu, ex.w13_t, ex.hidden, y.dtype)
        dx = torch.empty_like(dout)
        moe_dispatch_backward(drows, inv, k, dx)
        return dx, dw
