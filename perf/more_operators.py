"""The measured cases of the operators around the experts in nvfp4_mixture_experts_gb300: what a
block does before, between and after the experts' products, with activations held in 8 bits.

Five operators, in the order a step uses them:

  norm      h = x + residual, y = h / sqrt(mean h^2 + eps) * weight, y in its own type and as MXFP8
            (E4M3 elements, one power-of-two scale per 32), and its gradient
  route     scores of the experts (softmax or sigmoid), a bias for balance that steers the choice
            alone, groups of experts, top-k, renormalised weights; and the gradient of the logits
  quant8    MXFP8 quantisation of rows
  product8  grouped product of MXFP8 rows with MXFP4 weights, C_g = A_g . W_g^T
  swiglu    silu(gate) * up as MXFP8 rows for the next product, with a checkpoint of gate and up in
            8 bits; and the gradient that reads the checkpoint

Every case is a dict of plain values; prepare(case, seed) makes the inputs on the GPU, run(state)
is one pass -- through the library's calls where `own` is true, in elementary torch operations
where it is false -- and exact(case, seed) is the operator's definition in 64 bits.  MXFP8 results
are returned as float8 numbers and their power-of-two scales.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token before its layer: latency
        dict(name="norm_1_row", op="norm", back=False, T=1, H=4096, dtype="bf16", res=True, y=True,
             q=True, tiled=True, ld=0),
        # a prefill / training chunk: the residual stream, rows for the router in 16 bits and for
        # the products in 8
        dict(name="norm_8192", op="norm", back=False, T=8192, H=4096, dtype="bf16", res=True, y=True,
             q=True, tiled=True, ld=0),
        # the chunk's gradient, with the residual stream's own gradient added
        dict(name="norm_back_8192", op="norm", back=True, T=8192, H=4096, dtype="bf16", res=True, ld=0),
        # one decoded token of the 320-expert top-8 layer: latency
        dict(name="route_1_token", op="route", back=False, T=1, E=320, k=8, score="softmax", bias=False,
             groups=1, topg=1, top2=False, renorm=True, scale=1.0, dtype="fp32", ld=0),
        # a prefill chunk with sigmoid scores, a balancing bias and half of eight groups
        dict(name="route_8192_groups", op="route", back=False, T=8192, E=320, k=8, score="sigmoid",
             bias=True, groups=8, topg=4, top2=True, renorm=True, scale=2.5, dtype="fp32", ld=0),
        # a training chunk's gradient through softmax scores that are not renormalised: every
        # expert's logit has one
        dict(name="route_back_8192", op="route", back=True, T=8192, E=320, k=8, score="softmax",
             renorm=False, scale=1.0, dtype="fp32", ld=0),
        # a decode batch's rows: latency
        dict(name="quant8_64", op="quant8", rows=64, cols=4096, ceil=True, tiled=True, dtype="bf16"),
        # a training chunk's rows, or the gradients of its output
        dict(name="quant8_8192", op="quant8", rows=8192, cols=4096, ceil=True, tiled=True, dtype="bf16"),
        # the gate of a decode batch's expert rows, which are mostly padding
        dict(name="swiglu_64", op="swiglu", back=False, T=64, E=320, k=8, off=0, El=320, I=1280,
             ckpt=True, tiled=True, dtype="bf16"),
        # the gradient of a training chunk's gate from its 8-bit checkpoint
        dict(name="swiglu_back_8192", op="swiglu", back=True, T=8192, E=320, k=8, off=0, El=320, I=1280,
             ckpt=True, tiled=True, dtype="bf16"),
        # a decode batch's gate and up projections: most experts' weights are read for a few rows
        dict(name="product8_64", op="product8", T=64, N=2560, K=4096, E=320, off=0, El=320, k=8,
             out="bf16"),
        # a prefill chunk's gate and up projections, about 205 rows per expert
        dict(name="product8_8192", op="product8", T=8192, N=2560, K=4096, E=320, off=0, El=320, k=8,
             out="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "route", "quant8", "swiglu", "product8"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    ld = 0 if rng.random() < 0.7 else rng.randint(1, 24)
    if op == "norm":
        T, H = _log(rng, 1, 8192), _log(rng, 32, 8192)
        if rng.random() < 0.7:
            H = (H + 31) // 32 * 32
        T = max(1, min(T, 8192 * 4096 * 2 // (H * SIZE[dtype])))
        c = dict(op=op, back=rng.random() < 0.4, T=T, H=H, dtype=dtype, res=rng.random() < 0.7, ld=ld)
        if not c["back"]:
            c["q"] = H % 32 == 0 and rng.random() < 0.7
            c["y"] = not c["q"] or rng.random() < 0.5
            c["tiled"] = rng.random() < 0.6
        return c
    if op == "route":
        E = _log(rng, 8, 512)
        groups = 1
        if rng.random() < 0.5:
            groups = rng.choice((2, 4, 8))
            E = max(E // groups, 2) * groups
        topg = rng.randint(1, groups)
        k = rng.randint(1, min(8, E // groups * topg))
        c = dict(op=op, back=rng.random() < 0.4, T=_log(rng, 1, 8192), E=E, k=k,
                 score=rng.choice(("softmax", "sigmoid")), renorm=rng.random() < 0.6,
                 scale=rng.choice((1.0, 2.5)), dtype=rng.choice(("bf16", "fp16", "fp32", "fp32")), ld=ld)
        if c["back"]:
            c["k"] = max(2, k)  # (a single renormalised weight is constant)
        else:
            c.update(bias=rng.random() < 0.5, groups=groups, topg=topg, top2=rng.random() < 0.5)
        return c
    if op == "quant8":
        rows, cols = _log(rng, 1, 8192), (_log(rng, 1, 8192) + 31) // 32 * 32
        return dict(op=op, rows=max(1, min(rows, 8192 * 4096 // cols)), cols=cols, ceil=rng.random() < 0.5,
                    tiled=rng.random() < 0.6, dtype=dtype)
    E = _log(rng, 1, 320)
    k, T = rng.randint(1, min(8, E)), _log(rng, 1, 8192 if dtype != "fp32" else 4096)
    El = E if rng.random() < 0.6 else rng.randint(1, E)
    if T * k * El < 8 * E:  # (some pairs stay)
        El = E
    off = rng.randint(0, E - El)
    if op == "swiglu":
        return dict(op=op, back=rng.random() < 0.5, T=T, E=E,
                    k=k, off=off, El=El, I=(_log(rng, 32, 1280) + 31) // 32 * 32, ckpt=rng.random() < 0.7,
                    tiled=rng.random() < 0.6, dtype=dtype)
    N, K = _log(rng, 16, 4096), (_log(rng, 64, 4096) + 127) // 128 * 128
    if rng.random() < 0.7:
        N = (N + 7) // 8 * 8
    return dict(op=op, T=T, N=min(N, 2560 * 4096 // K), K=K, E=E, off=off, El=El, k=k,
                out=rng.choice(("bf16", "bf16", "fp16", "fp32")))


# ------------------------------------------------------------------------------- the inputs

def _rows(c, g):
    """counts [El], offsets [El + 1] and perm_src [cap] of tokens routed to k distinct experts of E
    each, uniform: the local pairs' rows by expert, each group's first row a multiple of 128; row r's
    entry is negative where the row is padding.  (Which pair a row holds is of no effect here.)"""
    T, k, E, El = c["T"], c["k"], c["E"], c["El"]
    ids = torch.randn(T, E, generator=g, device=DEV).topk(k, dim=1).indices.reshape(-1)
    counts = torch.bincount(ids, minlength=E)[c["off"]:c["off"] + El]
    offsets = torch.zeros(El + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum((counts + 127) // 128 * 128, 0)
    P = T * k
    cap = (P + min(El, P) * 127 + 127) // 128 * 128
    r = torch.arange(cap, device=DEV)
    e = (torch.searchsorted(offsets, r, right=True) - 1).clamp(0, El - 1)
    live = r - offsets[e] < counts[e]
    return counts.to(torch.int32), offsets.to(torch.int32), torch.where(live, r, -1).to(torch.int32), cap


def _strided(T, H, ld, dtype, g):
    x = torch.randn(T, H + ld, generator=g, device=DEV)
    # one channel in a hundred is an outlier, as in activations
    x.mul_(1 + 9.0 * (torch.rand(1, H + ld, generator=g, device=DEV) < 0.01))
    return x.to(dtype)[:, :H]


def _pow2(byte):
    """fp32 2^(byte - 127) of scale bytes 0..254 (integers), from the bits."""
    b = byte.to(torch.int32)
    return torch.where(b == 0, 0x400000, b << 23).view(torch.float32)


def _mx8(x, ceil):
    """MXFP8 of finite fp32 x [..., K]: (E4M3 elements [..., K] as float8, scale bytes [..., K / 32]).
    The scale of 32 elements is 2^e with e the exponent of their largest magnitude less 8 (that of 256,
    the largest power of two in E4M3), one more under the `ceil` rule where the largest magnitude would
    pass 448.  Elements round to the nearest E4M3 value, ties to the even code, and saturate at 448."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    bits = b.abs().amax(-1).view(torch.int32)
    s = (bits >> 23) - 8
    if ceil:
        s = s + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    s = s.clamp_min(0)
    v = (b * _pow2(254 - s)[..., None]).clamp(-448.0, 448.0)
    return v.reshape(x.shape).to(F8), s.to(torch.uint8)


def _tile_scales(sf):
    """Scale bytes [B, R, K / 32] -> the tiled layout of the product: 512-byte atoms, one per
    (128 rows, 4 scales), scale kk of row m at byte (m % 32) * 16 + (m / 32) * 4 + kk."""
    B, R, S = sf.shape
    RB, KA = (R + 127) // 128, (S + 3) // 4
    p = torch.zeros(B, RB * 128, KA * 4, dtype=torch.uint8, device=sf.device)
    p[:, :R, :S] = sf
    return p.view(B, RB, 4, 32, KA, 4).permute(0, 1, 4, 3, 2, 5).contiguous().view(-1)


def _sf_buffer(R, C, tiled):
    n = (R + 127) // 128 * ((C // 32 + 3) // 4) * 512 if tiled else R * C // 32
    return torch.zeros(n, dtype=torch.uint8, device=DEV)


def _u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device=DEV)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "norm":
        T, H, ld, dt = c["T"], c["H"], c["ld"], DTYPES[c["dtype"]]
        s["weight"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(dt)
        s["x"] = _strided(T, H, ld, dt, g)
        s["res"] = _strided(T, H, ld, dt, g) if c["res"] else None
        s["rstd"] = torch.empty(T, dtype=torch.float32, device=DEV)
        if c["back"]:  # the forward's h is `x` here, and `res` the gradient that h has from elsewhere
            h = s["x"].float()
            s["rstd"] = torch.rsqrt(h.square().mean(1) + EPS)
            s["dy"] = torch.randn(T, H, generator=g, device=DEV).to(dt)
            s["dx"] = torch.empty(T, H, dtype=dt, device=DEV)
            s["dw"] = torch.empty(H, dtype=torch.float32, device=DEV)
            s["ws"] = torch.empty(32 << 20, dtype=torch.uint8, device=DEV)
            return s
        s["h"] = torch.empty(T, H, dtype=dt, device=DEV) if c["res"] else None
        s["y"] = torch.empty(T, H, dtype=dt, device=DEV) if c["y"] else None
        s["codes"] = _u8(T, H) if c["q"] else None
        s["sf"] = _sf_buffer(T, H, c["tiled"]) if c["q"] else None
        return s
    if c["op"] == "route":
        T, E, k, ld = c["T"], c["E"], c["k"], c["ld"]
        s["logits"] = (torch.randn(T, E + ld, generator=g, device=DEV) * 1.5).to(DTYPES[c["dtype"]])[:, :E]
        if c["back"]:
            s["ids"] = torch.randn(T, E, generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32).contiguous()
            s["dw"] = torch.randn(T, k, generator=g, device=DEV)
            s["dlogits"] = torch.empty(T, E, dtype=s["logits"].dtype, device=DEV)
            return s
        s["bias"] = 0.05 * torch.randn(E, generator=g, device=DEV) if c["bias"] else None
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        s["w"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
        return s
    if c["op"] == "quant8":
        R, C = c["rows"], c["cols"]
        s["x"] = _strided(R, C, 0, DTYPES[c["dtype"]], g).contiguous()
        s["x"].mul_(torch.rand(R, 1, generator=g, device=DEV) >= 0.001)  # a row in a thousand is zero
        s["codes"], s["sf"] = _u8(R, C), _sf_buffer(R, C, c["tiled"])
        return s
    s["counts"], s["offsets"], s["perm"], s["cap"] = _rows(c, g)
    cap, live = s["cap"], s["perm"] >= 0
    if c["op"] == "swiglu":
        I, dt = c["I"], DTYPES[c["dtype"]]
        gu = torch.randn(cap, 2 * I, generator=g, device=DEV).mul_(1.5)
        if c["back"]:
            codes, sf = _mx8(gu, True)
            del gu
            # what no pair wrote is nobody's: NaN scales, never read into a result
            s["ckpt"], s["ckpt_sf"] = codes.view(torch.uint8), torch.where(live[:, None], sf, 255).contiguous()
            s["ds"] = torch.randn(cap, I, generator=g, device=DEV).to(dt)
            s["ds"][~live] = float("nan")
            s["codes"], s["sf"] = _u8(cap, 2 * I), _sf_buffer(cap, 2 * I, c["tiled"])
            return s
        s["gu"] = gu.to(dt)
        s["gu"][~live] = float("nan")
        s["codes"], s["sf"] = _u8(cap, I), _sf_buffer(cap, I, c["tiled"])
        s["ckpt"] = _u8(cap, 2 * I) if c["ckpt"] else None
        s["ckpt_sf"] = _u8(cap, 2 * I // 32) if c["ckpt"] else None
        return s
    N, K, El = c["N"], c["K"], c["El"]
    # the groups that have rows, and the largest one's rows: what the plain form's padded batch of
    # products is laid out by
    n = s["counts"].tolist()
    s["live"] = torch.tensor([i for i in range(El) if n[i]], dtype=torch.int64, device=DEV)
    s["most"] = max(n)
    codes, sf = _mx8(torch.randn(cap, K, generator=g, device=DEV), True)
    codes = codes.view(torch.uint8)
    codes[~live], sf[~live] = 0x7F, 255  # padding rows: stale, NaN elements and scales among them
    s["a_codes"], s["a_sf"] = codes, _tile_scales(sf[None])
    # random E2M1 codes under scales about those of weights ~ N(0, 0.02)
    s["w_codes"] = torch.randint(0, 256, (El, N, K // 2), dtype=torch.uint8, generator=g, device=DEV)
    w_sf = torch.randint(118, 121, (El, N, K // 32), dtype=torch.uint8, generator=g, device=DEV)
    s["w_sf"] = _tile_scales(w_sf)
    # rows that belong to no group stay as they are (zero); one row more than the capacity, where
    # the plain form puts the padding of its batch
    s["out"] = torch.zeros(cap + 1, N, dtype=DTYPES[c["out"]], device=DEV)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    v = torch.tensor((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0), device=DEV)
    v = torch.cat((v, -v))
    byte = torch.arange(256, device=DEV)
    s["lut"] = torch.stack((v[byte & 15], v[byte >> 4]), 1)   # the two values of a code byte
    return s


# ------------------------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _out8(codes, sf):
    return dict(codes=codes.view(F8), scales=sf.view(-1).view(E8))


def _run_own(s):
    import nvfp4_mixture_experts_gb300 as moe
    c = s["case"]
    layout = moe.MOE_SF_TILED if c.get("tiled") else moe.MOE_SF_CANONICAL
    if c["op"] == "norm":
        if c["back"]:
            moe.moe_rmsnorm_backward(s["dy"], s["x"], s["weight"], s["rstd"], s["dx"], s["dw"], s["ws"],
                                     dh=s["res"])
            return dict(dx=s["dx"], dw=s["dw"])
        moe.moe_rmsnorm(s["x"], s["weight"], EPS, residual=s["res"], h=s["h"], y=s["y"], rstd=s["rstd"],
                        codes=s["codes"], sf=s["sf"], sf_layout=layout)
        out = dict(h=s["h"], y=s["y"], rstd=s["rstd"])
        return {**out, **_out8(s["codes"], s["sf"])} if c["q"] else out
    if c["op"] == "route":
        score = moe.MOE_SCORE_SOFTMAX if c["score"] == "softmax" else moe.MOE_SCORE_SIGMOID
        if c["back"]:
            moe.moe_route_scores_backward(s["logits"], s["ids"], s["dw"], s["dlogits"], score=score,
                                          renormalise=c["renorm"], scale=c["scale"])
            return s["dlogits"]
        moe.moe_route_scores(s["logits"], s["ids"], s["w"], bias=s["bias"], score=score,
                             num_groups=c["groups"], topk_groups=c["topg"],
                             group_score=moe.MOE_GROUP_TOP2 if c["top2"] else moe.MOE_GROUP_MAX,
                             renormalise=c["renorm"], scale=c["scale"])
        return dict(ids=s["ids"], w=s["w"])
    if c["op"] == "quant8":
        moe.moe_quant_mxfp8(s["x"], s["codes"], s["sf"], layout,
                            scale_rule=moe.MOE_MX_CEIL if c["ceil"] else moe.MOE_MX_FLOOR)
        return _out8(s["codes"], s["sf"])
    if c["op"] == "swiglu":
        if c["back"]:
            moe.moe_swiglu_mxfp8_backward(s["ds"], s["ckpt"], s["ckpt_sf"], s["codes"], s["sf"], layout,
                                          perm_src=s["perm"])
            return _out8(s["codes"], s["sf"])
        moe.moe_swiglu_mxfp8(s["gu"], s["codes"], s["sf"], layout, ckpt=s["ckpt"], ckpt_sf=s["ckpt_sf"],
                             perm_src=s["perm"])
        out = _out8(s["codes"], s["sf"])
        return dict(s=out, ckpt=_out8(s["ckpt"], s["ckpt_sf"])) if c["ckpt"] else out
    out = s["out"][:s["cap"]]
    moe.moe_grouped_gemm_mxfp8(s["a_codes"], s["a_sf"], s["counts"], s["offsets"], s["w_codes"], s["w_sf"],
                               out, s["status"])
    return out


def _plain8(x, tiled, live=None, ceil=True):
    """x fp32 [R, C] as MXFP8 rows; rows that are not live are zero."""
    if live is not None:
        x = torch.where(live[:, None], x, 0.0)
    codes, sf = _mx8(x, ceil)
    if live is not None:
        sf = torch.where(live[:, None], sf, 0)
    return dict(codes=codes, scales=(_tile_scales(sf[None]) if tiled else sf.reshape(-1)).view(E8))


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        w = s["weight"].float()
        if c["back"]:
            h, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
            xh, d = h * rstd, dy * w
            dx = rstd * (d - xh * (d * xh).mean(1, keepdim=True))
            dx = dx + s["res"].float() if c["res"] else dx
            return dict(dx=dx.to(s["dy"].dtype), dw=(dy * xh).sum(0))
        h = (s["x"].float() + s["res"].float()).to(s["x"].dtype) if c["res"] else None
        hf = h.float() if c["res"] else s["x"].float()
        rstd = torch.rsqrt(hf.square().mean(1) + EPS)
        y = hf * rstd[:, None] * w
        out = dict(h=h, y=y.to(s["x"].dtype) if c["y"] else None, rstd=rstd)
        return {**out, **_plain8(y, c["tiled"])} if c["q"] else out
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        if c["back"]:
            l, ids, dw = s["logits"].float(), s["ids"].long(), s["dw"] * c["scale"]
            p = torch.sigmoid(l) if c["score"] == "sigmoid" else _softmax(l)
            ps = p.gather(1, ids)
            dp = dw
            if c["renorm"]:
                q = ps / ps.sum(1, keepdim=True)
                dp = (dw - (dw * q).sum(1, keepdim=True)) / ps.sum(1, keepdim=True)
            d = torch.zeros_like(p).scatter_add_(1, ids, dp)
            if c["score"] == "sigmoid":
                d = d * p * (1 - p)
            else:
                d = p * (d - (d * p).sum(1, keepdim=True))
            return d.to(s["logits"].dtype)
        # the choice in 64 bits: neighbouring keys lie as near as 32-bit rounding
        l = s["logits"].double()
        p = torch.sigmoid(l) if c["score"] == "sigmoid" else _softmax(l)
        key = p + s["bias"].double() if c["bias"] else p
        if c["groups"] > 1:
            by = key.view(T, c["groups"], -1)
            top = by.sort(dim=2, descending=True, stable=True).values
            gs = top[:, :, :2].sum(2) if c["top2"] else top[:, :, 0]
            order = gs.sort(dim=1, descending=True, stable=True).indices
            keep = torch.zeros(T, c["groups"], dtype=torch.bool, device=DEV)
            keep.scatter_(1, order[:, :c["topg"]], True)
            key = torch.where(keep[:, :, None], by, float("-inf")).view(T, E)
        ids = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
        w = p.gather(1, ids)
        w = w / w.sum(1, keepdim=True) if c["renorm"] else w
        return dict(ids=ids.to(torch.int32), w=(w * c["scale"]).float())
    if c["op"] == "quant8":
        return _plain8(s["x"].float(), c["tiled"], ceil=c["ceil"])
    if c["op"] == "swiglu":
        I, live = c["I"], s["perm"] >= 0
        if c["back"]:
            gu = s["ckpt"].view(F8).float().view(-1, 2 * I // 32, 32) * _pow2(s["ckpt_sf"])[..., None]
            gu, ds = gu.view(-1, 2 * I), s["ds"].float()
            g, u = gu[:, :I], gu[:, I:]
            q = torch.sigmoid(g)
            return _plain8(torch.cat((ds * u * q * (1 + g * (1 - q)), ds * g * q), 1), c["tiled"], live)
        gu = s["gu"].float()
        g, u = gu[:, :I], gu[:, I:]
        out = _plain8(g * torch.sigmoid(g) * u, c["tiled"], live)
        return dict(s=out, ckpt=_plain8(gu, False, live)) if c["ckpt"] else out
    N, K, cap = c["N"], c["K"], s["cap"]
    if s["most"] == 0:
        return s["out"][:cap]

    def scales(atoms, R):   # tiled scale bytes of matrices of R rows -> [B, R rounded up, K / 32]
        v = atoms.view(-1, (R + 127) // 128, (K // 32 + 3) // 4, 32, 4, 4).permute(0, 1, 4, 3, 2, 5)
        return v.reshape(v.shape[0], v.shape[1] * 128, -1)[..., :K // 32]

    # the groups as one padded batch
    i = torch.arange(s["most"], device=DEV)
    row = s["offsets"][s["live"]].long()[:, None] + i
    used = i < s["counts"][s["live"]][:, None]
    at = torch.where(used, row, 0)
    a = s["a_codes"].view(F8).float()[at].view(*at.shape, K // 32, 32) * _pow2(scales(s["a_sf"], cap)[0][at])[..., None]
    a = torch.where(used[..., None], a.view(*at.shape, K), 0.0)
    w = s["lut"][s["w_codes"][s["live"]].int()].view(-1, N, K // 32, 32)
    w = w.mul_(_pow2(scales(s["w_sf"], N)[s["live"]][:, :N])[..., None]).view(-1, N, K)
    s["out"][torch.where(used, row, cap)] = torch.bmm(a, w.transpose(1, 2)).to(s["out"].dtype)
    return s["out"][:cap]


def _softmax(l):
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


# ------------------------------------------------------------------------------- what it takes

def _kept(c):
    """Expected pairs of the shard: routing is uniform over the experts."""
    return c["T"] * c["k"] * c["El"] / c["E"]


def work(case):
    c = case
    mx = 1 + 1 / 32
    if c["op"] == "norm":
        n, es = c["T"] * c["H"], SIZE[c["dtype"]]
        if c["back"]:
            return {"bytes": n * es * (4 if c["res"] else 3) + 4 * c["T"] + c["H"] * (es + 4), "flops": 9 * n}
        per = es * (3 if c["res"] else 1) + es * c["y"] + mx * c["q"]
        return {"bytes": n * per + 4 * c["T"] + c["H"] * es, "flops": 6 * n}
    if c["op"] == "route":
        n, es, pairs = c["T"] * c["E"], SIZE[c["dtype"]], c["T"] * c["k"]
        if c["back"]:
            # only scores that are sums over all experts need every logit
            read = n if c["score"] == "softmax" and not c["renorm"] else pairs
            return {"bytes": (read + n) * es + 8 * pairs, "flops": 6 * n}
        return {"bytes": n * es + 8 * pairs + 4 * c["E"] * c["bias"], "flops": 4 * n}
    if c["op"] == "quant8":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (SIZE[c["dtype"]] + mx), "flops": 2 * n}
    P = _kept(c)
    if c["op"] == "swiglu":
        n, es = P * c["I"], SIZE[c["dtype"]]
        if c["back"]:
            return {"bytes": n * (es + 4 * mx), "flops": 16 * n}
        return {"bytes": n * (2 * es + mx + 2 * mx * c["ckpt"]), "flops": 10 * n}
    # experts that at least one token picked
    touched = c["El"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])
    return {"bytes": touched * c["N"] * c["K"] * (0.5 + 1 / 32) + P * c["K"] * mx + P * c["N"] * SIZE[c["out"]],
            "flops": 2 * P * c["N"] * c["K"]}


# ------------------------------------------------------------------------------- 64 bits

def _two_to(e):
    """2^e of whole numbers, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """Doubles rounded to the nearest E4M3 number, ties to the even one, at most 448: the spacing is
    2^(exponent - 3), at least 2^-9."""
    e = (torch.frexp(x).exponent - 1).clamp_min(-6)
    step = _two_to(e - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)   # (torch rounds halves to even)


def _exact8(x, tiled, live=None, ceil=True):
    """MXFP8 of doubles: the elements before their scales, and the scales, as doubles."""
    if live is not None:
        x = torch.where(live[:, None], x, torch.zeros_like(x))
    R, C = x.shape
    m = x.view(R, C // 32, 32).abs().amax(2)
    e = torch.frexp(m).exponent - 1 - 8
    if ceil:
        e = torch.where(m > 448 * _two_to(e), e + 1, e)
    e = torch.where(m > 0, e, -127).clamp(-127, 127)
    el = _e4m3(x.view(R, C // 32, 32) / _two_to(e)[..., None]).view(R, C)
    byte = (e + 127).to(torch.uint8)
    if tiled:
        r = torch.arange(R, device=DEV)[:, None]
        b = torch.arange(C // 32, device=DEV)[None, :]
        KA = (C // 32 + 3) // 4
        at = ((r // 128) * KA + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
        out = torch.zeros((R + 127) // 128 * KA * 512, dtype=torch.uint8, device=DEV)
        out[at] = byte
        byte = out
    return dict(codes=el, scales=_two_to(byte.reshape(-1).long() - 127))


def _decode8(codes, byte):
    """Doubles of E4M3 bytes [R, C] under scale bytes [R, C / 32], from the bits."""
    q = codes.long()
    mant, ex = q & 7, (q >> 3) & 15
    v = torch.where(ex == 0, mant * 2.0 ** -9, (8 + mant) * _two_to(ex - 10))
    return torch.where(q >= 128, -v, v) * _two_to(byte.long() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    c = case
    s = prepare(c, seed)
    if c["op"] == "norm":
        w = s["weight"].double()
        if c["back"]:
            h, dy, r = s["x"].double(), s["dy"].double(), s["rstd"].double()[:, None]
            dot = torch.einsum("th,h,th->t", dy, w, h)[:, None] / c["H"]
            dx = r * dy * w - h * r ** 3 * dot
            return dict(dx=dx + s["res"].double() if c["res"] else dx, dw=torch.einsum("th,th,ti->h", dy, h, r))
        h = s["x"].double()
        if c["res"]:
            h = (h + s["res"].double()).to(s["x"].dtype).double()   # h is what its type holds
        rstd = 1 / torch.sqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / c["H"] + EPS)
        y = torch.einsum("th,t,h->th", h, rstd, w)
        out = dict(h=h if c["res"] else None, y=y if c["y"] else None, rstd=rstd)
        return {**out, **_exact8(y, c["tiled"])} if c["q"] else out
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        l = s["logits"].double()
        logp = -torch.log1p(torch.exp(-l)) if c["score"] == "sigmoid" else l - torch.logsumexp(l, 1, keepdim=True)
        p = torch.exp(logp)
        if c["back"]:
            # w_j = scale p_j, or scale p_j / sum p: the derivative with respect to every logit
            ids = s["ids"].long()
            q = p.gather(1, ids)
            S = q.sum(1, keepdim=True)
            dw = s["dw"].double() * c["scale"]
            hit = torch.zeros(T, E, dtype=torch.float64, device=DEV).scatter_(1, ids, 1.0)
            per = torch.zeros_like(hit).scatter_(1, ids, dw)              # dw of the chosen
            mean = (dw * q).sum(1, keepdim=True) / S
            if c["score"] == "sigmoid":
                return (per - mean * hit) * p * (1 - p) / S if c["renorm"] else per * p * (1 - p)
            # softmax renormalised over the chosen is the softmax of the chosen logits
            return (per - mean * hit) * p / S if c["renorm"] else p * (per - mean * S)
        key = p + (s["bias"].double() if c["bias"] else 0.0)
        n = E // c["groups"]
        if c["groups"] > 1:
            top = key.view(T, c["groups"], n).topk(min(2, n), dim=2).values
            gs = top.sum(2) if c["top2"] else top[..., 0]
            # a group is out where topg others are before it: better, or as good with a lower index
            i = torch.arange(c["groups"], device=DEV)
            before = (gs[:, None, :] > gs[:, :, None]) | ((gs[:, None, :] == gs[:, :, None]) & (i[None, :] < i[:, None]))
            out = before.sum(2) >= c["topg"]
            key = torch.where(out.repeat_interleave(n, 1), -math.inf, key)
        ids = []
        for _ in range(k):  # the first of the largest, k times
            ids.append((key == key.amax(1, keepdim=True)).int().argmax(1))
            key = key.scatter(1, ids[-1][:, None], -math.inf)
        ids = torch.stack(ids, 1)
        w = logp.gather(1, ids)
        w = torch.exp(w - torch.logsumexp(w, 1, keepdim=True)) if c["renorm"] else torch.exp(w)
        return dict(ids=ids.to(torch.int32), w=w * c["scale"])
    if c["op"] == "quant8":
        return _exact8(s["x"].double(), c["tiled"], ceil=c["ceil"])
    if c["op"] == "swiglu":
        I, live = c["I"], s["perm"] >= 0
        if s["cap"] * I > 1 << 28:
            return None  # (its doubles would fill the card)
        if c["back"]:
            gu = torch.where(live[:, None], _decode8(s["ckpt"], s["ckpt_sf"]), 0.0)
            ds = torch.where(live[:, None], s["ds"].double(), 0.0)
            g, u = gu[:, :I], gu[:, I:]
            e = torch.exp(-g)
            # silu(g) = g / (1 + e^-g)
            dg = ds * u * (1 + e + g * e) / (1 + e) ** 2
            return _exact8(torch.cat((dg, ds * g / (1 + e)), 1), c["tiled"], live)
        gu = torch.where(live[:, None], s["gu"].double(), 0.0)
        out = _exact8(gu[:, :I] / (1 + torch.exp(-gu[:, :I])) * gu[:, I:], c["tiled"], live)
        return dict(s=out, ckpt=_exact8(gu, False, live)) if c["ckpt"] else out
    if _kept(c) * c["N"] * c["K"] * 2 > 8e12:
        return None
    N, K, KA = c["N"], c["K"], (c["K"] // 32 + 3) // 4
    out = torch.zeros(s["cap"], N, dtype=torch.float64, device=DEV)

    def bytes_of(atoms, row0, R):
        """[R, K / 32] scale bytes of the rows from row0 of the atoms."""
        r = torch.arange(row0, row0 + R, device=DEV)[:, None]
        b = torch.arange(K // 32, device=DEV)[None, :]
        return atoms[((r // 128) * KA + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]

    per = (N + 127) // 128 * KA * 512
    for i, (n, o) in enumerate(zip(s["counts"].tolist(), s["offsets"].tolist())):
        if n:
            q = torch.empty(N, K, dtype=torch.int64, device=DEV)
            q[:, 0::2], q[:, 1::2] = s["w_codes"][i].long() & 15, s["w_codes"][i].long() >> 4
            mant, ex = q & 1, (q >> 1) & 3                           # E2M1: subnormal 0 and 1/2
            v = torch.where(ex == 0, 0.5 * mant, (1 + 0.5 * mant) * _two_to(ex - 1))
            v = torch.where(q >= 8, -v, v)
            v = v * _two_to(bytes_of(s["w_sf"][i * per:(i + 1) * per], 0, N).long() - 127).repeat_interleave(32, 1)
            out[o:o + n] = _decode8(s["a_codes"][o:o + n], bytes_of(s["a_sf"], o, n)) @ v.t()
    return out
