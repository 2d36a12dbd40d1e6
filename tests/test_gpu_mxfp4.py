"""MXFP4 quantisation, scale layout and the grouped product against plain 64-bit implementations.

Tolerances: every step of the quantiser is exact or a single rounding to a code, so codes, scales
and values are equal.  The product's terms are exact and its fp32 sums of K terms, in any order
and even truncated, are within K 2^-23 of the sum of the terms' magnitudes; then one rounding."""
import numpy as np
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
import ops_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F = 2.0 ** -23


def f64(t):
    return t.detach().cpu().double().numpy()


def u8(n, fill=0):
    return torch.full((n,), fill, dtype=torch.uint8, device="cuda")


def matrix(rows, cols, dtype, seed):
    """Values over a wide range of magnitudes, with zero blocks, ties and the type's extremes."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-12, 12, (rows, 1))
    x[rng.random((rows, cols)) < 0.2] = 0.0
    ties = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.5, 7.5, -0.25, -5.0, -0.0], (rows, cols))
    pick = rng.random((rows, cols)) < 0.3
    x[pick] = (ties * 2.0 ** rng.integers(-3, 4, (rows, 1)))[pick]
    t = torch.from_numpy(x).to(DT[dtype])
    info = torch.finfo(DT[dtype])
    t.view(-1)[0] = info.max
    t.view(-1)[-1] = -info.tiny
    if rows * cols > 64:
        t.view(-1)[rows * cols // 2] = info.smallest_normal / 4 if dtype == "fp32" else info.tiny
    return t


def as_type(v, dtype):
    """fp64 values rounded once to the type (overflow to infinity), as fp64."""
    return torch.from_numpy(v).to(DT[dtype]).double().numpy()


def check_quant(x, dtype, ceil, layout, transpose=False, perm=None):
    """x: CPU [B, R, C] (any strides) of the dtype."""
    xd = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)
    B, R, C = x.shape
    R2, C2 = (C, R) if transpose else (R, C)
    codes = u8(B * R2 * C2 // 2, 0xA5)
    sf = u8(moe.moe_mxfp4_scale_bytes(B, R2, C2, layout), 0xA5)
    vals = torch.full((B, R2, C2), -3.0, dtype=x.dtype, device="cuda")
    pd = None if perm is None else torch.from_numpy(perm).cuda()
    moe.moe_quant_mxfp4(xd, codes, sf, layout, transpose=transpose,
                        scale_rule=moe.MOE_MX_CEIL if ceil else moe.MOE_MX_FLOOR, perm_src=pd,
                        values=vals)
    gc, gs = codes.cpu().numpy().reshape(B, R2, C2 // 2), sf.cpu().numpy().reshape(B, -1)
    for b in range(B):
        m = x[b].double().numpy()
        c, s, v = ref.quant_mxfp4(m.T if transpose else m, ceil)
        live = np.ones(R2, bool) if perm is None else perm >= 0
        assert np.array_equal(gc[b][live], ref.pack(c)[live])
        assert np.all(gc[b][~live] == 0xA5)
        if layout == moe.MOE_SF_CANONICAL:
            got = gs[b].reshape(R2, C2 // 32)
            assert np.array_equal(got[live], s[live])
        else:
            want = ref.tile_scales(s, fill=0xA5)
            if perm is not None:
                at = ref.tile_scales(np.where(live[:, None], 1, 0).repeat(C2 // 32, 1), fill=0)
                want, got = want[at == 1], gs[b][at == 1]
            else:
                got = gs[b]
            assert np.array_equal(got, want)
        got = f64(vals[b])
        assert np.array_equal(got[live], as_type(v, dtype)[live], equal_nan=True)
        assert np.all(got[~live] == -3.0)


SHAPES = [(1, 1, 32), (1, 3, 96), (2, 130, 160), (1, 257, 4096), (3, 7, 8224)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,R,C", SHAPES)
def test_quantiser(B, R, C, dtype):
    for i, (ceil, layout) in enumerate([(False, 0), (True, 1), (False, 1)]):
        check_quant(torch.stack([matrix(R, C, dtype, 10 * i + b) for b in range(B)]), dtype, ceil, layout)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,R,C", [(1, 32, 1), (2, 96, 33), (1, 160, 130), (2, 4128, 65), (1, 64, 1000)])
def test_quantiser_of_the_transpose(B, R, C, dtype):
    for i, (ceil, layout) in enumerate([(True, 0), (False, 1)]):
        check_quant(torch.stack([matrix(R, C, dtype, 10 * i + b) for b in range(B)]), dtype, ceil,
                    layout, transpose=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,R,C,pad", [(1, 4100, 1056, 0), (3, 1001, 1504, 8), (1, 516, 8224, 1),
                                       (1, 4097, 1024, 0)])
def test_quantiser_of_large_matrices(B, R, C, pad, dtype):
    """Rows that end inside a warp's run, and rows of no pair, in matrices of many runs."""
    perm = np.arange(R, dtype=np.int32)
    perm[R // 3::7] = -1
    x = torch.zeros(B, R, C + pad, dtype=DT[dtype])[:, :, :C]
    for b in range(B):
        x[b] = matrix(R, C, dtype, b)
    check_quant(x, dtype, False, moe.MOE_SF_TILED, perm=perm if B == 1 else None)
    check_quant(x, dtype, True, moe.MOE_SF_CANONICAL)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("pad", [1, 8, 16])
def test_strided_input(dtype, transpose, pad):
    base = torch.zeros(2, 67, 128 + pad, dtype=DT[dtype])
    view = base[:, 2:66, :128]
    for b in range(2):
        view[b] = matrix(64, 128, dtype, b)
    check_quant(view, dtype, False, moe.MOE_SF_TILED, transpose=transpose)


def test_unaligned_input():
    flat = torch.zeros(1 + 64 * 64, dtype=torch.bfloat16, device="cuda")
    x = flat[1:].view(64, 64)
    m = matrix(64, 64, "bf16", 4)
    x.copy_(m)
    codes, sf = u8(64 * 32), u8(64 * 2)
    moe.moe_quant_mxfp4(x, codes, sf, moe.MOE_SF_CANONICAL)
    c, s, _ = ref.quant_mxfp4(m.double().numpy(), False)
    assert np.array_equal(codes.cpu().numpy().reshape(64, 32), ref.pack(c))
    assert np.array_equal(sf.cpu().numpy().reshape(64, 2), s)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_infinities_and_nans_give_nan_blocks(dtype, transpose):
    x = matrix(64, 64, dtype, 3)
    for at, v in (((3, 40), float("inf")), ((10, 5), float("nan")), ((11, 63), float("-inf"))):
        x[at] = v
    check_quant(x[None], dtype, False, moe.MOE_SF_TILED, transpose=transpose)


def test_smallest_magnitudes():
    x = torch.zeros(4, 32)
    x[0, 3] = 2.0 ** -149
    x[1, 4] = -(2.0 ** -126)
    x[2, :8] = torch.tensor([1.0, 2, 3, 4, 5, 6, 7, 8]) * 2.0 ** -130
    for ceil in (False, True):
        check_quant(x[None], "fp32", ceil, moe.MOE_SF_CANONICAL)


def test_rows_of_no_pair_are_skipped():
    perm = np.full(300, -1, np.int32)
    perm[[0, 1, 2, 128, 131, 256, 299]] = [5, 6, 0, 1, 2, 3, 4]
    x = torch.stack([matrix(300, 288, "bf16", 9)])
    x[0][torch.from_numpy(perm < 0)] = float("nan")
    check_quant(x, "bf16", False, moe.MOE_SF_TILED, perm=perm)


@pytest.mark.parametrize("B,R,C", [(1, 1, 32), (2, 130, 160), (3, 256, 4096), (1, 300, 96)])
def test_tile_scales(B, R, C):
    rng = np.random.default_rng(R)
    sf = rng.integers(0, 256, (B, R, C // 32)).astype(np.uint8)
    out = u8(moe.moe_mxfp4_scale_bytes(B, R, C, moe.MOE_SF_TILED), 0xA5)
    moe.moe_mxfp4_tile_scales(torch.from_numpy(sf).cuda(), B, R, C, out)
    want = np.concatenate([ref.tile_scales(s) for s in sf])
    assert np.array_equal(out.cpu().numpy(), want)


# ------------------------------------------------------------------ the product

def operand(rng, rows, K, spread=6):
    codes = rng.integers(0, 16, (rows, K))
    sf = rng.integers(127 - spread, 127 + spread + 1, (rows, K // 32))
    return codes, sf


def run_product(counts, N, K, dtype, seed=0, ld=0, ws=True, grouped=True, offsets=None, cap=None,
                mutate=None):
    """Random operands; returns (out as fp64, reference, magnitudes, per-row group or -1, status)."""
    rng = np.random.default_rng(seed)
    G = len(counts)
    if offsets is None:
        offsets = np.concatenate([[0], np.cumsum([(c + 127) // 128 * 128 for c in counts])])
    cap = int(offsets[-1]) if cap is None else cap
    a_codes, a_sf = operand(rng, cap, K)
    w = [operand(rng, N, K) for _ in range(G)]
    group = np.full(cap, -1)
    for g, c in enumerate(counts):
        group[offsets[g]:offsets[g] + c] = g
    a_codes[group < 0], a_sf[group < 0] = 7, 255     # rows of no group: NaN scales
    if mutate:
        mutate(a_codes, a_sf, w)
    out = torch.full((cap, N + ld), -3.0, dtype=DT[dtype], device="cuda")[:, :N]
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32).cuda()  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = moe.moe_mxfp4_workspace_size(cap, G, N, K)
    moe.moe_grouped_gemm_mxfp4(
        torch.from_numpy(ref.pack(a_codes)).cuda(),
        torch.from_numpy(ref.tile_scales(a_sf, fill=255)).cuda(),
        i32(counts) if grouped else None, i32(offsets) if grouped else None,
        torch.from_numpy(np.stack([ref.pack(c) for c, _ in w])).cuda(),
        torch.from_numpy(np.concatenate([ref.tile_scales(s, fill=255) for _, s in w])).cuda(),
        out, u8(need, 0xFF) if ws else None, status)
    want, mag = np.full((cap, N), -3.0), np.zeros((cap, N))
    av = ref.decode(a_codes, a_sf)
    for g in range(G):
        rows = group == g
        wv = ref.decode(*w[g])
        want[rows] = av[rows] @ wv.T
        mag[rows] = np.abs(av[rows]) @ np.abs(wv).T
    return f64(out), want, mag, group, status.item()


def check_product(counts, N, K, dtype, **kw):
    got, want, mag, group, status = run_product(counts, N, K, dtype, **kw)
    assert status == 0
    live = group >= 0
    assert np.all(got[~live] == -3.0), "rows of no group are left as they are"
    ok = ref.rounded_ok(got[live], want[live], K * F * mag[live], dtype)
    assert np.all(ok), (np.argwhere(~ok)[:4], got[live][~ok][:4], want[live][~ok][:4])


PRODUCTS = [  # counts, N, K
    ([1], 128, 32), ([1], 1, 64), ([3], 130, 96), ([128], 256, 256), ([129], 256, 128),
    ([257], 384, 512), ([0, 5, 0, 0, 1], 64, 160), ([0, 0], 64, 64), ([16, 17, 32, 33, 64, 65], 200, 352),
    ([1] * 40, 256, 1024), ([300, 2, 255, 256, 1], 136, 288), ([130] * 9, 640, 96),
    ([5, 0, 700, 31], 512, 2048), ([2, 1], 2560, 4096), ([8], 72, 8192),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("counts,N,K", PRODUCTS, ids=[str(i) for i in range(len(PRODUCTS))])
def test_product(counts, N, K, dtype):
    if dtype == "fp16":   # keep the sums in fp16's range
        check_product(counts, N, K, dtype, mutate=lambda a, s, w: [x.__isub__(8) for _, x in w])
    else:
        check_product(counts, N, K, dtype, seed=len(counts))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ld", [1, 4, 8])
def test_product_strided_output_and_no_workspace(dtype, ld):
    check_product([20, 140, 1], 200, 288, dtype, ld=ld)
    check_product([20, 140, 1], 200, 288, dtype, ld=ld, ws=False)
    check_product([1], 333, 4096, dtype, ld=ld, ws=False)


@pytest.mark.parametrize("rows", [1, 127, 300])
def test_product_of_one_group(rows):
    check_product([rows], 160, 224, "bf16", grouped=False, cap=rows)


def test_groups_need_not_be_packed():
    check_product([3, 130, 7], 96, 128, "fp32", offsets=[0, 256, 640, 900], cap=900)


def test_last_group_may_end_at_the_capacity():
    check_product([128, 2], 96, 128, "fp32", offsets=[0, 128, 256], cap=130)


def test_repeated_calls_agree_bit_for_bit():
    a = run_product([1, 3, 2], 512, 4096, "fp32", seed=4)[0]
    for _ in range(3):
        assert np.array_equal(a, run_product([1, 3, 2], 512, 4096, "fp32", seed=4)[0])


def test_bad_groups_are_skipped_and_flagged():
    got, want, mag, group, status = run_product([4, 4], 64, 64, "fp32", offsets=[0, 128, 256])
    assert status == 0
    # a start that is no multiple of 128, and a group past the capacity
    for counts, offs in (([4, 4], [0, 64, 256]), ([4, 200], [0, 128, 256])):
        out = torch.full((256, 64), -3.0, device="cuda")
        i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        moe.moe_grouped_gemm_mxfp4(u8(256 * 32).view(256, 32), u8(1024, 127), i32(counts), i32(offs),
                                   u8(2 * 64 * 32).view(2, 64, 32), u8(1024, 127), out, None, st)
        assert st.item() == moe.MOE_DEV_BAD_INDEX
        assert torch.all(out[:4] == 0.0) and torch.all(out[4:] == -3.0)


def test_nan_scales_reach_their_rows_and_columns_only():
    def mutate(a_codes, a_sf, w):
        a_sf[5, 1] = 255
        w[0][1][9, 0] = 255
        a_codes[5, 32:64], w[0][0][9, :32] = 2, 2   # nonzero codes under the NaN scales
        a_codes[:, :32] = np.where(a_codes[:, :32] % 8 == 0, 1, a_codes[:, :32])
        w[0][0][:, 32:64] = np.where(w[0][0][:, 32:64] % 8 == 0, 1, w[0][0][:, 32:64])

    got, want, mag, group, status = run_product([20], 64, 128, "fp32", mutate=mutate)
    live = group >= 0
    bad = np.isnan(got[live])
    assert np.array_equal(bad, np.isnan(want[live]))
    assert bad[5].all() and bad[:, 9].all() and bad.sum() == 64 + 20 - 1


def test_extreme_scales():
    """Scales at both ends whose products are representable."""
    def mutate(a_codes, a_sf, w):
        a_sf[:] = 250
        for c, s in w:
            s[:] = 3
    check_product([33], 64, 64, "fp32", mutate=mutate)


def test_product_of_quantised_rows_and_its_gradient():
    """x -> quantise -> product; the gradient with respect to the quantised rows is the product
    of the output's gradient with the transposed weights."""
    torch.manual_seed(0)
    M, N, K = 70, 96, 160
    x, wt = torch.randn(M, K, device="cuda"), torch.randn(1, N, K, device="cuda") * 0.1
    dout = torch.randn(M, N, device="cuda")

    def quant(t, transpose=False):
        B = t.shape[0] if t.dim() == 3 else 1
        R, C = t.shape[-2:][::-1] if transpose else t.shape[-2:]
        codes = u8(B * R * C // 2).view((B, R, C // 2) if t.dim() == 3 else (R, C // 2))
        sf = u8(moe.moe_mxfp4_scale_bytes(B, R, C, moe.MOE_SF_TILED))
        vals = torch.empty((*t.shape[:-2], R, C), device="cuda")
        moe.moe_quant_mxfp4(t, codes, sf, moe.MOE_SF_TILED, transpose=transpose, values=vals)
        return codes, sf, vals

    xc, xs, xv = quant(x)
    wc, ws, wv = quant(wt)
    out = torch.empty(M, N, device="cuda")
    moe.moe_grouped_gemm_mxfp4(xc, xs, None, None, wc, ws, out)
    want, mag = f64(xv) @ f64(wv[0]).T, np.abs(f64(xv)) @ np.abs(f64(wv[0])).T
    assert np.all(ref.rounded_ok(f64(out), want, K * F * mag, "fp32"))
    dc, ds, dv = quant(dout)
    tc, ts, tv = quant(wt, transpose=True)
    dx = torch.empty(M, K, device="cuda")
    moe.moe_grouped_gemm_mxfp4(dc, ds, None, None, tc, ts, dx)
    want, mag = f64(dv) @ f64(tv[0]).T, np.abs(f64(dv)) @ np.abs(f64(tv[0])).T
    assert np.all(ref.rounded_ok(f64(dx), want, N * F * mag, "fp32"))


def test_products_gradient_is_the_difference():
    """With weights that both quantisations hold exactly, out is linear in the rows, so for any two
    sets of representable rows L(A2) - L(A1) = <dL/dA, A2 - A1>, L = <dout, out>."""
    rng = np.random.default_rng(5)
    M, N, K = 40, 96, 160
    grid = np.array([-4.0, -2.0, -1.0, 0.0, 1.0, 2.0, 4.0])

    def exact(rows, cols):   # every block has the largest magnitude 4: scale 1, codes exact
        m = rng.choice(grid, (rows, cols))
        m[:, ::32], m[::32, :] = 4.0, -4.0
        return torch.from_numpy(m).float().cuda()

    def quant(t, transpose=False):
        R, C = (t.shape[1], t.shape[0]) if transpose else t.shape
        codes, sf = u8(R * C // 2).view(R, C // 2), u8(moe.moe_mxfp4_scale_bytes(1, R, C, moe.MOE_SF_TILED))
        moe.moe_quant_mxfp4(t, codes, sf, moe.MOE_SF_TILED, transpose=transpose)
        return codes, sf

    def product(a, w, rows, cols):
        out = torch.empty(rows, cols, device="cuda")
        moe.moe_grouped_gemm_mxfp4(*a, None, None, w[0][None], w[1], out)
        return out

    w = exact(N, K)
    a1, a2, dout = exact(M, K), exact(M, K), exact(M, N)
    loss = [float((f64(dout) * f64(product(quant(a), quant(w), M, N))).sum()) for a in (a1, a2)]
    grad = f64(product(quant(dout), quant(w, transpose=True), M, K))
    # every sum is of integers below 2^24: exact in fp32
    assert loss[1] - loss[0] == (grad * (f64(a2) - f64(a1))).sum()


def test_offsets_past_two_to_the_31():
    """Outputs and inputs of over 2^32 elements: the last rows are where they belong."""
    cap, N, K = (1 << 20) + 128, 4128, 32
    a = u8(cap * 16).view(cap, 16)
    a[1 << 20:].fill_(0x22)                      # every element 1
    sf = u8(moe.moe_mxfp4_scale_bytes(1, cap, K, moe.MOE_SF_TILED), 127)
    w, wsf = u8(N * 16, 0x44).view(1, N, 16), u8(moe.moe_mxfp4_scale_bytes(1, N, K, moe.MOE_SF_TILED), 127)
    out = torch.zeros(cap, N, dtype=torch.bfloat16, device="cuda")
    i32 = lambda v: torch.tensor([v], dtype=torch.int32).cuda()  # noqa: E731
    moe.moe_grouped_gemm_mxfp4(a, sf, i32(5), i32(1 << 20), w, wsf, out)
    assert torch.all(out[(1 << 20):(1 << 20) + 5] == 64.0)      # 32 products 1 x 2
    assert torch.all(out[(1 << 20) + 5:] == 0) and torch.all(out[(1 << 20) - 64:1 << 20] == 0)
    # the quantiser reads that matrix and its transpose
    x = out[:, :4096]
    codes = u8(cap * 2048)
    moe.moe_quant_mxfp4(x, codes, u8(moe.moe_mxfp4_scale_bytes(1, cap, 4096, 0)), 0)
    got = codes.view(cap, 2048)
    assert torch.all(got[(1 << 20):(1 << 20) + 5] == 0x66)      # 64 = 4 x 2^4
    assert torch.all(got[(1 << 20) + 5:] == 0) and torch.all(got[:64] == 0)
    tcodes = u8(4096 * cap // 2)
    moe.moe_quant_mxfp4(x, tcodes, u8(moe.moe_mxfp4_scale_bytes(1, 4096, cap, 0)), 0, transpose=True)
    got = tcodes.view(4096, cap // 2)
    assert torch.all(got[:, 1 << 19:(1 << 19) + 2] == 0x66) and torch.all(got[:, (1 << 19) + 2] == 0x06)
    assert torch.all(got[:, (1 << 19) + 3:] == 0) and torch.all(got[:, :64] == 0)


def test_another_stream_orders_quantiser_and_product():
    M, N, K = 384, 256, 512
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x = torch.zeros(M, K, device="cuda")
        w = torch.ones(1, N, K, device="cuda")
        codes, wc = u8(M * K // 2).view(M, K // 2), u8(N * K // 2).view(1, N, K // 2)
        sf = u8(moe.moe_mxfp4_scale_bytes(1, M, K, moe.MOE_SF_TILED))
        ws = u8(moe.moe_mxfp4_scale_bytes(1, N, K, moe.MOE_SF_TILED))
        out = torch.empty(M, N, device="cuda")
        for i in range(1, 5):             # each call must see the one before it
            x += 1.0
            moe.moe_quant_mxfp4(w, wc, ws, moe.MOE_SF_TILED)
            moe.moe_quant_mxfp4(x, codes, sf, moe.MOE_SF_TILED)
            moe.moe_grouped_gemm_mxfp4(codes, sf, None, None, wc, ws, out)
        total = out.sum()
    side.synchronize()
    assert total.item() == 4.0 * K * M * N


def test_calls_replay_in_a_graph():
    M, N, K = 100, 200, 256
    x, w = torch.randn(M, K, device="cuda"), torch.randn(1, N, K, device="cuda")
    codes, wc = u8(M * K // 2).view(M, K // 2), u8(N * K // 2).view(1, N, K // 2)
    sf = u8(moe.moe_mxfp4_scale_bytes(1, M, K, moe.MOE_SF_TILED))
    ws = u8(moe.moe_mxfp4_scale_bytes(1, N, K, moe.MOE_SF_TILED))
    out = torch.empty(M, N, device="cuda")

    def step():
        moe.moe_quant_mxfp4(w, wc, ws, moe.MOE_SF_TILED)
        moe.moe_quant_mxfp4(x, codes, sf, moe.MOE_SF_TILED)
        moe.moe_grouped_gemm_mxfp4(codes, sf, None, None, wc, ws, out)

    step()
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x.mul_(2.0)                           # twice the rows: the same codes, scales one up
    g.replay()
    assert torch.equal(out, 2 * first)
