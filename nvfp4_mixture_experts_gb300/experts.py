"""MXExperts: a shard of gated experts with frozen MXFP4 weights, forward and backward.

The handle-free operators in the order a training step (or a forward that wants gradients later)
calls them:

  forward   moe_dispatch -> moe_quant_mxfp4 -> moe_grouped_gemm_mxfp4 (gate_up) -> silu(g) * u
            -> moe_quant_mxfp4 -> moe_grouped_gemm_mxfp4 (down) -> moe_combine_weighted
  backward  moe_combine_backward -> moe_quant_mxfp4 -> product with W2^T -> the gate's gradient
            -> moe_quant_mxfp4 -> product with W13^T -> moe_dispatch_backward

With act_bits 8 the activations and gradients are MXFP8 instead, and the gate's own operators hold
what the backward pass needs of gate and up in 8 bits:

  forward   moe_dispatch -> moe_quant_mxfp8 -> moe_grouped_gemm_mxfp8 (gate_up) -> moe_swiglu_mxfp8
            -> moe_grouped_gemm_mxfp8 (down) -> moe_combine_weighted
  backward  moe_combine_backward -> moe_quant_mxfp8 -> product with W2^T
            -> moe_swiglu_mxfp8_backward -> product with W13^T -> moe_dispatch_backward

MXShared is the same gate and products on every token: the shared expert.

The quantisation of activations and gradients is passed straight through; the weights (adapters
and routers train around them) have no gradient, and the gradients have none (second derivatives
raise).  With act_bits 4 the elementwise gate is torch's, on all rows of
the sorted buffers: rows of no pair hold stale values that nothing downstream reads.
"""
import torch

from . import (MOE_DEV_WAIT_TIMEOUT, MOE_ERR_DEVICE_STATUS, MOE_ERR_INVALID, MOE_ERR_TIMEOUT,
               MOE_ERR_UNSUPPORTED, MOE_MX_CEIL, MOE_OK, MOE_SF_TILED, MoEError, moe_combine_backward,
               moe_combine_weighted, moe_dispatch, moe_dispatch_backward,
               moe_dispatch_rows_capacity, moe_grouped_gemm_mxfp4, moe_grouped_gemm_mxfp8,
               moe_mxfp4_scale_bytes, moe_mxfp4_tile_scales, moe_quant_mxfp4, moe_quant_mxfp8,
               moe_swiglu_mxfp8, moe_swiglu_mxfp8_backward)

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


def _empty8(rows, cols, device):
    """Room for an MXFP8 matrix [rows, cols] with tiled scales."""
    codes = torch.empty(rows, cols, dtype=torch.uint8, device=device)
    return codes, torch.empty(moe_mxfp4_scale_bytes(1, rows, cols, MOE_SF_TILED), dtype=torch.uint8,
                              device=device)


def as_rows(t):
    """t [rows, cols] itself where its rows are contiguous and apart, else a copy (of a transposed tensor, or of
    one row that is broadcast)."""
    return t if t.stride(1) == 1 and t.stride(0) >= t.shape[1] else t.contiguous()


def quantise8(x, perm_src=None):
    """(codes, tiled scales) of the rows x [rows, cols] as an MXFP8 matrix."""
    codes, sf = _empty8(*x.shape, x.device)
    moe_quant_mxfp8(x, codes, sf, MOE_SF_TILED, perm_src=perm_src)
    return codes, sf


def _held(dtype):
    """The type in which gate and up, and the gradient of their product, lie between a product and the gate, for
    tokens of a type.  It is theirs (the gate rounds to 8 bits with a scale for 32 elements, so 16 bits lose
    nothing that counts), but for fp16: its range would make an infinity of a value past 65504, and the gate NaN
    of the row."""
    return torch.float32 if dtype == torch.float16 else dtype


class _Gated8:
    """silu(gate) * up between two products of MXFP8 rows with MXFP4 weights, and its gradient.  counts,
    offsets, perm: the rows' groups (None: one group, of all rows)."""

    def __init__(self, ex, counts=None, offsets=None, perm=None):
        self.ex, self.groups, self.perm = ex, (counts, offsets), perm

    def product(self, a, w, cols, dtype):
        out = torch.empty(a[0].shape[0], cols, dtype=dtype, device=a[0].device)
        moe_grouped_gemm_mxfp8(*a, *self.groups, *w, out, status=self.ex.status)
        return out

    def forward(self, a, dtype, keep):
        """a: the rows' codes and tiled scales; (rows of the down product, checkpoint or None)."""
        ex, rows, dev = self.ex, a[0].shape[0], a[0].device
        gu = self.product(a, ex.w13, 2 * ex.inter, _held(dtype))
        s, ckpt = _empty8(rows, ex.inter, dev), (None, None)
        if keep:
            ckpt = (torch.empty(rows, 2 * ex.inter, dtype=torch.uint8, device=dev),
                    torch.empty(rows, ex.inter // 16, dtype=torch.uint8, device=dev))
        moe_swiglu_mxfp8(gu, *s, MOE_SF_TILED, ckpt=ckpt[0], ckpt_sf=ckpt[1], perm_src=self.perm)
        return self.product(s, ex.w2, ex.hidden, dtype), ckpt

    def backward(self, dy, ckpt):
        """The gradient of the rows for the gradient dy of the down product's."""
        ex = self.ex
        if ex.w13_t is None:
            raise RuntimeError("%s without transposed weights has no backward" % type(ex).__name__)
        ds = self.product(quantise8(dy, self.perm), ex.w2_t, ex.inter, _held(dy.dtype))
        dgu = _empty8(dy.shape[0], 2 * ex.inter, dy.device)
        moe_swiglu_mxfp8_backward(ds, *ckpt, *dgu, MOE_SF_TILED, perm_src=self.perm)
        return self.product(dgu, ex.w13_t, ex.hidden, dy.dtype)


class MXExperts:
    """Experts local_off .. local_off + num_local - 1 of num_experts: w13 [num_local, 2I, H] (gate
    rows, then up rows) and w2 [num_local, H, I], H and I multiples of 32 (with act_bits 8, of 128)."""

    def __init__(self, num_experts, local_off, w13, w13_sf, w2, w2_sf, w13_t=None, w2_t=None,
                 act_bits=4):
        """w13, w2: MXFP4 codes [num_local, rows, cols / 2] with tiled scales w13_sf, w2_sf.  w13_t,
        w2_t: (codes, scales) of each expert's transposed matrices; without them there is no
        backward.  act_bits: of the activations and gradients that the products read (4 or 8)."""
        self.num_experts, self.local_off = num_experts, local_off
        self.num_local, two_inter, half_hidden = w13.shape
        self.hidden, self.inter = 2 * half_hidden, two_inter // 2
        self.act_bits = act_bits
        if act_bits not in (4, 8):
            raise MoEError(MOE_ERR_INVALID, "MXExperts: act_bits %r" % (act_bits,))
        if act_bits == 8 and (self.hidden % 128 or self.inter % 128):
            raise MoEError(MOE_ERR_UNSUPPORTED, "MXExperts: hidden %d, inter %d with 8-bit activations"
                           % (self.hidden, self.inter))
        self.w13, self.w2, self.w13_t, self.w2_t = (w13, w13_sf), (w2, w2_sf), w13_t, w2_t
        self.status = torch.zeros(1, dtype=torch.int32, device=w13.device)

    @classmethod
    def from_master(cls, num_experts, local_off, w13, w2, backward=True, act_bits=4):
        """Quantises bf16/fp16/fp32 master weights; for the backward pass their transposes too
        (blocks of 32 run along the contraction, so a transpose has its own codes)."""
        return cls(num_experts, local_off, *quantise(w13), *quantise(w2),
                   quantise(w13, transpose=True) if backward else None,
                   quantise(w2, transpose=True) if backward else None, act_bits=act_bits)

    @classmethod
    def from_checkpoint(cls, num_experts, local_off, w13, w13_sf, w2, w2_sf, act_bits=4):
        """Codes and canonical scales [num_local, rows, cols / 32] of a checkpoint (forward only)."""
        tiled = []
        for codes, sf in ((w13, w13_sf), (w2, w2_sf)):
            n, rows, cols = codes.shape[0], codes.shape[1], codes.shape[2] * 2
            t = torch.empty(moe_mxfp4_scale_bytes(n, rows, cols, MOE_SF_TILED), dtype=torch.uint8,
                            device=codes.device)
            moe_mxfp4_tile_scales(sf, n, rows, cols, t)
            tiled += [codes, t]
        return cls(num_experts, local_off, *tiled, act_bits=act_bits)

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


class MXShared(MXExperts):
    """The shared expert: MXFP4 weights w13 [1, 2I, H] and w2 [1, H, I] applied to every token with 8-bit
    activations.  Made as MXExperts are, from_master(w13, w2) or from_checkpoint(w13, w13_sf, w2, w2_sf)."""

    def __init__(self, num_experts, local_off, *args, **kw):
        super().__init__(num_experts, local_off, *args, **dict(kw, act_bits=8))
        if self.num_local != 1:
            raise MoEError(MOE_ERR_INVALID, "MXShared: %d experts" % self.num_local)

    @classmethod
    def from_master(cls, w13, w2, backward=True):
        return super().from_master(1, 0, w13, w2, backward=backward, act_bits=8)

    @classmethod
    def from_checkpoint(cls, w13, w13_sf, w2, w2_sf):
        return super().from_checkpoint(1, 0, w13, w13_sf, w2, w2_sf, act_bits=8)

    def __call__(self, x, eight=None):
        """[T, H] in x's type for tokens x [T, H]; differentiable in x.  eight: x as an MXFP8 matrix with
        tiled scales, where the caller has it already (moe_rmsnorm's)."""
        if eight is not None and tuple(eight[0].shape) != tuple(x.shape):
            raise MoEError(MOE_ERR_INVALID, "MXShared: codes %s of rows %s" % (tuple(eight[0].shape), tuple(x.shape)))
        return _Shared.apply(x, *(eight or (None, None)), self)


class _FirstOrder(torch.autograd.Function):
    """Gradients that are part of a graph (create_graph) and have no gradient of their own; name: whose."""

    @staticmethod
    def forward(ctx, name, *grads):
        ctx.name = name
        return tuple(g.clone() for g in grads)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("%s has no second derivatives" % ctx.name)


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

        w = topk_w.detach().float().contiguous()
        out = torch.empty(T, ex.hidden, dtype=dt, device=dev)
        if ex.act_bits == 8:
            gated = _Gated8(ex, counts, offsets, perm)
            y, ckpt = gated.forward(quantise8(rows, perm), dt, any(ctx.needs_input_grad))
            moe_combine_weighted(y, inv, w, out)
            ctx.ex, ctx.gated, ctx.k = ex, gated, k
            ctx.save_for_backward(y, w, inv, *ckpt)
            return out

        def product(a, w, cols, dtype):
            out = torch.empty(cap, cols, dtype=dtype, device=dev)
            moe_grouped_gemm_mxfp4(*quantise(a, perm_src=perm), counts, offsets, *w, out,
                                   status=ex.status)
            return out

        gu = product(rows, ex.w13, 2 * ex.inter, torch.float32)
        gate, up = gu[:, :ex.inter], gu[:, ex.inter:]
        y = product(torch.nn.functional.silu(gate) * up, ex.w2, ex.hidden, dt)
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
            grads = _FirstOrder.apply("MXExperts", *(g.requires_grad_() for g in grads))
        return (*grads, None, None)

    @staticmethod
    def gradients(ctx, dout):
        ex, k = ctx.ex, ctx.k
        if ex.w13_t is None:
            raise RuntimeError("MXExperts without transposed weights has no backward")
        if ex.act_bits == 8:
            y, w, inv, *ckpt = ctx.saved_tensors
            dout = dout.to(y.dtype).contiguous()
            dy, dw = torch.empty_like(y), torch.empty_like(w)
            moe_combine_backward(dout, y, inv, w, dy, dw)
            dx = torch.empty_like(dout)
            moe_dispatch_backward(ctx.gated.backward(dy, ckpt), inv, k, dx)
            return dx, dw
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


class _Shared(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, codes, sf, ex):
        gated = _Gated8(ex)
        eight = quantise8(as_rows(x)) if codes is None else (codes, sf)
        y, ckpt = gated.forward(eight, x.dtype, ctx.needs_input_grad[0])
        ctx.gated, ctx.dtype = gated, x.dtype
        ctx.save_for_backward(*ckpt)
        return y

    @staticmethod
    def backward(ctx, dout):
        with torch.no_grad():
            dx = ctx.gated.backward(dout.to(ctx.dtype).contiguous(), ctx.saved_tensors)
        if torch.is_grad_enabled():
            dx, = _FirstOrder.apply("MXShared", dx.requires_grad_())
        return dx, None, None, None
