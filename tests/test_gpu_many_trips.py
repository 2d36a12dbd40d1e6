"""The handle-free operators at sizes where every warp, block or CTA pair takes several pieces of the
work one after another, as a prompt's do: state that is carried or alternates from one to the next.

References are in 64 bits on the GPU, or the same call on pieces that are small enough for one piece
each (the other tests compare those with plain implementations).  Tolerances: a sum of n terms in
fp32 is within n 2^-23 of the sum of the terms' magnitudes, then one rounding to the type."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
STEP = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24, "fp32": 2.0 ** -149}
F = 2.0 ** -23


def i32(*shape):
    return torch.full(shape, -7, dtype=torch.int32, device="cuda")


def u8(n, fill=0xA5):
    return torch.full((n,), fill, dtype=torch.uint8, device="cuda")


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def near(got, want, slack, kind):
    """Within `slack`, the error before the last rounding, and one rounding to `kind`."""
    return (got.double() - want).abs() <= UNIT[kind] * (want.abs() + slack) + slack + STEP[kind]


def route(T, E, k, g):
    return torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int().contiguous()


def maps(ids, off, El, align, cap):
    """The sort's definition with torch's stable sort, on 64-bit numbers."""
    le = ids.reshape(-1).long() - off
    key = torch.where((le >= 0) & (le < El), le, El)
    order = torch.argsort(key, stable=True)
    n = torch.bincount(key, minlength=El + 1)
    first = torch.cumsum(n, 0) - n
    offsets = torch.zeros(El + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum((n[:El] + align - 1) // align * align, 0)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(order.numel(), device="cuda")
    inv = torch.where(key < El, offsets[key] + rank - first[key], -1)
    perm = torch.full((cap,), -1, dtype=torch.int64, device="cuda")
    live = inv >= 0
    perm[inv[live]] = torch.nonzero(live)[:, 0]
    return n[:El], offsets, perm, inv


def dispatch(x, ids, E, off, El, align):
    T, k = ids.shape
    cap = moe.moe_dispatch_rows_capacity(T, k, El, align)
    o = dict(counts=i32(El), offsets=i32(El + 1), perm=i32(cap), inv=i32(T * k), cap=cap, rows=None)
    if x is not None:
        o["rows"] = torch.full((cap, x.shape[1]), -3.0, dtype=x.dtype, device="cuda")
    moe.moe_dispatch(x, ids, E, off, El, align, o["counts"], o["offsets"], o["perm"], o["inv"], o["rows"])
    return o


# more than 8 batches of 32 pairs a warp from 131073 pairs
@pytest.mark.parametrize("T,E,k,off,El,align", [(70001, 320, 2, 0, 320, 1), (40009, 320, 8, 160, 160, 128),
                                                (131073, 7, 1, 0, 7, 4), (40009, 1024, 32, 3, 1000, 1)])
def test_sort_of_many_pairs(T, E, k, off, El, align):
    ids = route(T, E, k, generator(T)) if E >= k else None
    o = dispatch(None, ids, E, off, El, align)
    counts, offsets, perm, inv = maps(ids, off, El, align, o["cap"])
    for name, want in (("counts", counts), ("offsets", offsets), ("perm", perm), ("inv", inv)):
        assert torch.equal(o[name].long(), want), name


# T, H, k, E, off, El, ld: by tokens and rows' bytes, each form of the row mover, of combine and of
# its gradient, with more tokens (or runs of them) than the grid has warps or blocks
ROWS = [(20011, 40, 3, 12, 2, 9, 0),      # gradient: one warp a token
        (20011, 41, 3, 12, 0, 12, 1),
        (10007, 3080, 3, 12, 2, 9, 0),    # two warps a token, four pairs at a time
        (10007, 2504, 6, 12, 2, 9, 8),    # two warps, all pairs at once
        (5003, 4104, 9, 12, 0, 12, 0),
        (40003, 24, 1, 6, 1, 4, 0),       # several tokens a warp or block
        (19999, 3080, 1, 6, 1, 4, 0),
        (40003, 24, 2, 6, 0, 6, 0),
        (10001, 3080, 2, 6, 1, 4, 3)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,k,E,off,El,ld", ROWS)
def test_rows_of_many_tokens(T, H, k, E, off, El, ld, dtype):
    g, dt = generator(T + H), DT[dtype]
    H = H if dtype != "fp32" else (H + 1) // 2     # the same bytes
    def tokens(fill=None):  # noqa: E306
        t = torch.randn(T, H + ld, generator=g, device="cuda") if fill is None else \
            torch.full((T, H + ld), fill, device="cuda")
        return t.to(dt)[:, :H]
    x, ids = tokens(), route(T, E, k, g)
    o = dispatch(x, ids, E, off, El, 1)
    _, _, perm, inv = maps(ids, off, El, 1, o["cap"])
    assert torch.equal(o["inv"].long(), inv) and torch.equal(o["perm"].long(), perm)
    live = perm >= 0
    assert torch.equal(o["rows"][live], x[perm[live] // k]) and torch.all(o["rows"][~live] == -3.0)

    y = torch.randn(o["cap"], H, generator=g, device="cuda").to(dt)
    y[~live] = float("nan")
    w = torch.rand(T, k, generator=g, device="cuda") + 0.1
    w[inv.view(T, k) < 0] = float("nan")
    out, dx = tokens(float("nan")), tokens(float("nan"))
    moe.moe_combine_weighted(y, o["inv"], w, out)
    moe.moe_dispatch_backward(y, o["inv"], k, dx)
    dout = tokens()
    dy, dw = torch.full_like(y, -3.0), torch.full_like(w, -3.0)
    moe.moe_combine_backward(dout, y, o["inv"], w, dy, dw)
    assert torch.all(dy[~live] == -3.0)

    sums = torch.zeros(4, T, H, dtype=torch.float64, device="cuda")
    iv = inv.view(T, k)
    for j in range(k):
        t = torch.nonzero(iv[:, j] >= 0)[:, 0]
        r, wj = iv[t, j], w[t, j].double()[:, None]
        v, d = y[r].double(), dout[t].double()
        for i, term in enumerate((v, v.abs(), v * wj, (v * wj).abs())):
            sums[i].index_add_(0, t, term)
        dots = d * v
        assert torch.all((dw[t, j].double() - dots.sum(1)).abs() <= (H + 2) * F * dots.abs().sum(1) + 1e-40)
        assert torch.all(near(dy[r], d * wj, F * (d * wj).abs(), dtype))
    assert torch.all(dw[iv < 0] == 0.0)
    assert torch.all(near(dx, sums[0], (k + 1) * F * sums[1], dtype))
    assert torch.all(near(out, sums[2], (k + 1) * F * sums[3], dtype))


# ------------------------------------------------------------------ the product

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def values(codes, sf):
    """fp64 values of packed codes [..., K / 2] and canonical scales [..., K / 32]."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device="cuda")
    c = codes.long()
    v = torch.stack((table[c & 15], table[c >> 4]), -1).flatten(-2)
    return v * torch.exp2(sf.double() - 127).repeat_interleave(32, -1)


def operand(B, R, K, g):
    """Codes [B, R, K / 2], canonical scales [B, R, K / 32] and their tiled form."""
    codes = torch.randint(0, 256, (B, R, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sf = torch.randint(122, 128, (B, R, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    tiled = u8(moe.moe_mxfp4_scale_bytes(B, R, K, moe.MOE_SF_TILED))
    moe.moe_mxfp4_tile_scales(sf, B, R, K, tiled)
    return codes, sf, tiled


# rows of the groups: up to 64 (the small stages), and over it
FEW = [1, 33, 0, 64, 2, 31, 32, 50, 17, 5, 0, 48] * 9
MANY = [1, 300, 32, 0, 257, 33, 128, 64, 200, 513, 2, 255, 96, 31, 256, 160, 65, 7] * 3


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("counts,N,K", [(FEW, 1000, 96), (FEW, 640, 1056), (MANY, 1288, 64), (MANY, 1031, 352),
                                        (MANY, 1024, 2080)], ids=range(5))
def test_product_of_many_tiles(counts, N, K, dtype):
    """Several tiles a CTA pair, of mixed sizes: both accumulators, those that overlap and those that
    do not, and the ring's phases from tile to tile."""
    tiles = sum((c + 255) // 256 for c in counts) * ((N + 255) // 256)
    assert tiles > 2 * 76
    g = generator(N + K)
    offs, at = [], 0
    for c in counts:
        offs.append(at)
        at += (c + 127) // 128 * 128
    a, sa, ta = operand(1, at, K, g)
    w, sw, tw = operand(len(counts), N, K, g)
    out = torch.full((at, N), -3.0, dtype=DT[dtype], device="cuda")
    status = torch.zeros_like(i32(1))
    to_i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for _ in range(2):                                   # the second time as the first
        moe.moe_grouped_gemm_mxfp4(a[0], ta, to_i32(counts), to_i32(offs), w, tw, out, status=status)
    assert status.item() == 0
    av = values(a[0], sa[0])
    for i, (c, o) in enumerate(zip(counts, offs)):
        wv = values(w[i], sw[i])
        want, mag = av[o:o + c] @ wv.t(), av[o:o + c].abs() @ wv.abs().t()
        if dtype == "fp16":
            assert float(want.abs().max() if c else 0) < 65504
        assert torch.all(near(out[o:o + c], want, K * F * mag, dtype)), i
        end = offs[i + 1] if i + 1 < len(offs) else at
        assert torch.all(out[o + c:end] == -3.0)


# ------------------------------------------------------------------ the quantiser

def quantise(x, layout, transpose, ceil):
    B, R, C = x.shape
    rows, cols = (C, R) if transpose else (R, C)
    codes = u8(B * rows * cols // 2).view(B, rows, cols // 2)
    sf = u8(moe.moe_mxfp4_scale_bytes(B, rows, cols, layout))
    vals = torch.full((B, rows, cols), -3.0, dtype=x.dtype, device="cuda")
    moe.moe_quant_mxfp4(x, codes, sf, layout, transpose=transpose,
                        scale_rule=moe.MOE_MX_CEIL if ceil else moe.MOE_MX_FLOOR, values=vals)
    return codes, sf, vals


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,R,C,transpose,piece", [
    (1, 40000, 1024, False, 4000),      # long rows: 19456 warps, a run of 1024 elements each
    (2, 12001, 2080, False, 1500),
    (1, 262144, 32, False, 32768),      # short rows: 622592 threads, eight elements each
    (3, 30001, 160, False, 6000),
    (1, 4096, 20001, True, 1000),       # 2432 blocks, a tile of 128 x 128 (x 64) elements each
    (7, 2592, 4104, True, 500),
])
def test_quantiser_of_many_pieces(B, R, C, transpose, piece, dtype):
    g = generator(R + C)
    x = torch.randn(B, R, C, generator=g, device="cuda")
    x = (x * torch.exp2(torch.randint(-6, 7, (B, R, 1), generator=g, device="cuda").float())).to(DT[dtype])
    n = C if transpose else R           # rows of the result
    k = R if transpose else C
    for ceil in (False, True):
        codes, sf, vals = quantise(x, moe.MOE_SF_CANONICAL, transpose, ceil)
        sf = sf.view(B, n, k // 32)
        for b in range(B):
            for r in range(0, n, piece):
                part = x[b:b + 1, :, r:r + piece] if transpose else x[b:b + 1, r:r + piece]
                c, s, v = quantise(part, moe.MOE_SF_CANONICAL, transpose, ceil)
                m = c.shape[1]
                assert torch.equal(codes[b, r:r + m], c[0]) and torch.equal(vals[b, r:r + m], v[0])
                assert torch.equal(sf[b, r:r + m].flatten(), s)
        codes2, tiled, vals2 = quantise(x, moe.MOE_SF_TILED, transpose, ceil)
        assert torch.equal(codes2, codes) and torch.equal(vals2, vals)
        # the tiled layout, its rows past the end left out
        KA, RB = (k // 32 + 3) // 4, (n + 127) // 128
        t = tiled.view(B, RB, KA, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(B, RB * 128, KA * 4)
        assert torch.equal(t[:, :n, :k // 32], sf) and not torch.any(t[:, :n, k // 32:])
        again = u8(tiled.numel())
        moe.moe_mxfp4_tile_scales(sf.contiguous(), B, n, k, again)
        a = again.view(B, RB, KA, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(B, RB * 128, KA * 4)
        assert torch.equal(a[:, :n], t[:, :n]) and not torch.any(a[:, n:])
