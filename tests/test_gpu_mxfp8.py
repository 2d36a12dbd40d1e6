"""MXFP8 rows: the quantiser, the gate with its 8-bit checkpoint and gradient, and the grouped product
with MXFP4 weights, against 64-bit implementations."""
import numpy as np
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
import ops8_ref as ref
import ops_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CANON, TILED = moe.MOE_SF_CANONICAL, moe.MOE_SF_TILED


def u8(*shape, fill=0):
    return torch.full(shape, fill, dtype=torch.uint8, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


def scales(sf, R, C, layout):
    s = sf.cpu().numpy()
    return s.reshape(R, C // 32) if layout == CANON else ref.untile(s, R, C // 32)


def sf_for(R, C, layout, fill=0):
    return u8(moe.moe_mxfp4_scale_bytes(1, R, C, layout), fill=fill)


# ------------------------------------------------------------------------------- quantiser

@pytest.mark.parametrize("R,C", [(1, 32), (3, 96), (130, 160), (700, 64), (5, 4096), (257, 2080), (1100, 1056)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", [CANON, TILED])
@pytest.mark.parametrize("ceil", [False, True])
def test_quantiser(R, C, dtype, layout, ceil):
    g = torch.Generator("cuda").manual_seed(R)
    x = torch.randn(R, C + 8, generator=g, device="cuda")
    x *= torch.exp(4 * torch.randn(R, 1, generator=g, device="cuda"))
    x[0, :32] = 0
    x[R // 2, 5], x[R - 1, 40 % C] = -0.0, 449.0
    x = x.to(DT[dtype])[:, :C]
    codes, sf, values = u8(R, C), sf_for(R, C, layout, 9), torch.empty(R, C, device="cuda").to(DT[dtype])
    moe.moe_quant_mxfp8(x, codes, sf, layout, scale_rule=moe.MOE_MX_CEIL if ceil else moe.MOE_MX_FLOOR,
                        values=values)
    c, s, v = ref.quant_mxfp8(f64(x), ceil)
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(scales(sf, R, C, layout), s)
    ok = np.isfinite(torch.from_numpy(v).to(DT[dtype]).double().numpy())   # (fp16: values past 65504)
    assert np.array_equal(f64(values)[ok], torch.from_numpy(v).to(DT[dtype]).double().numpy()[ok])


@pytest.mark.parametrize("ceil", [False, True])
def test_quantiser_on_borders(ceil):
    """Every E4M3 number, every midpoint of two and its neighbours; scales at their ends; NaN and infinity."""
    m = ref.E4M3_MAG
    mid = ((m[1:] + m[:-1]) / 2).astype(np.float32)
    v = np.concatenate([m, mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9)), [449, 480, 511]])
    v = np.concatenate([v, -v])
    v = np.pad(v, (0, -len(v) % 31)).reshape(-1, 31)
    big = np.where(np.abs(v).max(1) > 448, 256.0, 448.0)[:, None]      # the block's scale is 2^0, or as it falls
    x = np.concatenate([v, big], 1).astype(np.float32)
    tiny = np.float32(2.0) ** -np.arange(100, 149)
    ends = np.zeros((60, 32), np.float32)
    ends[:49, 0], ends[:49, 3] = tiny, -tiny / 3
    ends[49, 2], ends[50, 1], ends[51, 31] = np.nan, np.inf, -np.inf
    ends[52, :2], ends[53, 0], ends[54, 0] = 3e38, 1.75 * 2.0 ** 40, np.nextafter(np.float32(1.75 * 2.0 ** 40), np.float32(1e20))
    x = np.concatenate([x, ends])
    R = x.shape[0]
    codes, sf, values = u8(R, 32), u8(R), torch.empty(R, 32, device="cuda")
    moe.moe_quant_mxfp8(torch.from_numpy(x).cuda(), codes, sf, CANON,
                        scale_rule=moe.MOE_MX_CEIL if ceil else moe.MOE_MX_FLOOR, values=values)
    c, s, val = ref.quant_mxfp8(x.astype(np.float64), ceil)
    assert np.array_equal(sf.cpu().numpy(), s.reshape(-1)) and np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(f64(values), val, equal_nan=True)


def test_quantiser_batches_padding_and_tiled_scales():
    x = torch.randn(3, 130, 96, device="cuda").bfloat16()
    codes, sf = u8(3, 130, 96), u8(3 * 130 * 3)
    moe.moe_quant_mxfp8(x, codes, sf, CANON)
    for b in range(3):
        c, s, _ = ref.quant_mxfp8(f64(x[b]), True)
        assert np.array_equal(codes[b].cpu().numpy(), c)
        assert np.array_equal(sf.view(3, 130, 3)[b].cpu().numpy(), s)
    tiled, again = u8(3 * 2 * 512), u8(3 * 2 * 512)
    moe.moe_quant_mxfp8(x, codes, tiled, TILED)
    moe.moe_mxfp4_tile_scales(sf, 3, 130, 96, again)
    for b in range(3):
        assert np.array_equal(ref.untile(tiled.view(3, -1)[b].cpu().numpy(), 130, 4),
                              ref.untile(again.view(3, -1)[b].cpu().numpy(), 130, 4))
    perm = torch.arange(130, dtype=torch.int32, device="cuda")
    perm[::3] = -1
    c2, s2 = u8(130, 96, fill=5), u8(130 * 3, fill=6)
    moe.moe_quant_mxfp8(x[0], c2, s2, CANON, perm_src=perm)
    dead = (perm < 0).cpu()
    assert torch.all(c2.cpu()[dead] == 5) and torch.all(s2.view(130, 3).cpu()[dead] == 6)
    assert torch.equal(c2.cpu()[~dead], codes[0].cpu()[~dead])


# ------------------------------------------------------------------------------- the gate

# sigmoid: two instructions within 2^-22 and the exponent's rounding (|g| <= 20 here), then two products
GATE_TOL = 2 * 2.0 ** -22 + 20 * 2.0 ** -23 + 2 * 2.0 ** -24
# a gradient's terms: 1 + g (1 - s) is a sum of terms of at most 1 + |g|, each within GATE_TOL of itself
GATES = [(1, 32), (3, 96), (130, 64), (257, 160), (40, 1280), (9, 4096)]


def live_rows(R, g):
    perm = torch.arange(R, dtype=torch.int32)
    if R > 2:
        perm[torch.randperm(R, generator=g)[:R // 3]] = -1
    return perm.cuda()


@pytest.mark.parametrize("R,I", GATES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", [CANON, TILED])
def test_gate(R, I, dtype, layout):
    g = torch.Generator().manual_seed(I)
    pad = {"bf16": 8, "fp16": 3, "fp32": 0}[dtype]
    gu = (torch.randn(R, 2 * I + pad, generator=g) * 2).clamp(-20, 20).to(DT[dtype]).cuda()[:, :2 * I]
    perm = live_rows(R, g)
    live = (perm >= 0).cpu().numpy()
    gu[~torch.from_numpy(live)] = float("nan")
    for p in (perm, None):
        for ceil in (True, False):
            codes, sf, ck, ck_sf = u8(R, I, fill=3), sf_for(R, I, layout, 4), u8(R, 2 * I, fill=5), u8(R * I // 16, fill=6)
            rule = moe.MOE_MX_CEIL if ceil else moe.MOE_MX_FLOOR
            moe.moe_swiglu_mxfp8(gu, codes, sf, layout, ckpt=ck, ckpt_sf=ck_sf, perm_src=p, scale_rule=rule)
            x = f64(gu)[live]
            c, s, _ = ref.quant_mxfp8(x, ceil)
            assert np.array_equal(ck.cpu().numpy()[live], c)
            assert np.array_equal(ck_sf.view(R, -1).cpu().numpy()[live], s)
            want = ref.swiglu(x[:, :I], x[:, I:])
            sc = scales(sf, R, I, layout)
            assert ref.mx8_close(codes.cpu().numpy()[live], sc[live], want, GATE_TOL, ceil)
            if p is not None:
                assert np.all(codes.cpu().numpy()[~live] == 3) and np.all(ck.cpu().numpy()[~live] == 5)
                assert np.all(sc[~live] == 4) and np.all(ck_sf.view(R, -1).cpu().numpy()[~live] == 6)
            else:
                assert np.all(sc[~live] == 255) and np.all(codes.cpu().numpy()[~live] == 0)
            if layout == TILED and (I // 32) % 4:
                assert np.all(ref.untile(sf.cpu().numpy(), R, (I // 32 + 3) // 4 * 4)[live][:, I // 32:] == 0)
            c2, s2 = u8(R, I, fill=3), sf_for(R, I, layout, 4)
            moe.moe_swiglu_mxfp8(gu, c2, s2, layout, perm_src=p, scale_rule=rule)   # no checkpoint
            assert torch.equal(c2, codes) and torch.equal(s2, sf)


@pytest.mark.parametrize("R,I", GATES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", [CANON, TILED])
def test_gate_gradient(R, I, dtype, layout):
    g = torch.Generator().manual_seed(I + 1)
    gu = (torch.randn(R, 2 * I, generator=g) * 2).clamp(-20, 20).cuda()
    ck, ck_sf = u8(R, 2 * I), u8(R * I // 16)
    moe.moe_quant_mxfp8(gu, ck, ck_sf, CANON)
    pad = {"bf16": 8, "fp16": 3, "fp32": 0}[dtype]
    ds = torch.randn(R, I + pad, generator=g).to(DT[dtype]).cuda()[:, :I]
    perm = live_rows(R, g)
    live = (perm >= 0).cpu().numpy()
    held = ref.decode8(ck.cpu().numpy(), ck_sf.view(R, -1).cpu().numpy())[live]
    ds[~torch.from_numpy(live)] = float("nan")
    ck[~torch.from_numpy(live)] = 127
    gate, up, d = held[:, :I], held[:, I:], f64(ds)[live]
    dg, du = ref.swiglu_grad(d, gate, up)
    want = np.concatenate([dg, du], 1)
    s = ref.sigmoid(gate)
    slack = 4 * GATE_TOL * np.concatenate([np.abs(d * up) * s * (1 + np.abs(gate)), np.abs(d * gate) * s], 1)
    codes, sf = u8(R, 2 * I, fill=3), sf_for(R, 2 * I, layout, 4)
    out = torch.full((R, 2 * I), 7.0, device="cuda").to(DT[dtype])
    moe.moe_swiglu_mxfp8_backward(ds, ck, ck_sf, codes, sf, layout, perm_src=perm, dgate_up=out)
    assert np.all(ops_ref.rounded_ok(f64(out)[live], want, slack, dtype))
    assert np.all(f64(out)[~live] == 7)
    sc = scales(sf, R, 2 * I, layout)
    # of a block's largest: its terms against its result
    m = np.abs(want).reshape(-1, 2 * I // 32, 32).max(-1)
    worst = float((slack.reshape(-1, 2 * I // 32, 32).max(-1) / np.maximum(m, 1e-30)).max())
    assert worst < 1e-2
    assert ref.mx8_close(codes.cpu().numpy()[live], sc[live], want, worst)
    assert np.all(codes.cpu().numpy()[~live] == 3) and np.all(sc[~live] == 4)
    c2, s2 = u8(R, 2 * I, fill=3), sf_for(R, 2 * I, layout, 4)
    moe.moe_swiglu_mxfp8_backward(ds, ck, ck_sf, c2, s2, layout, perm_src=perm)
    o2 = torch.full((R, 2 * I), 7.0, device="cuda").to(DT[dtype])
    moe.moe_swiglu_mxfp8_backward(ds, ck, ck_sf, perm_src=perm, dgate_up=o2)
    assert torch.equal(c2, codes) and torch.equal(s2, sf) and torch.equal(o2, out)


def test_gate_gradient_against_differences():
    rng = np.random.default_rng(4)
    gu = rng.normal(size=(2, 64))
    ck, ck_sf = u8(2, 64), u8(4)
    moe.moe_quant_mxfp8(torch.from_numpy(gu).float().cuda(), ck, ck_sf, CANON)
    held = ref.decode8(ck.cpu().numpy(), ck_sf.view(2, 2).cpu().numpy())
    ds = rng.normal(size=(2, 32)).astype(np.float32).astype(np.float64)
    out = torch.empty(2, 64, device="cuda")
    moe.moe_swiglu_mxfp8_backward(torch.from_numpy(ds).float().cuda(), ck, ck_sf, dgate_up=out)
    num = np.zeros_like(held)
    for i in np.ndindex(held.shape):
        e = np.zeros_like(held)
        e[i] = 1e-5
        f = lambda a: (ref.swiglu(a[:, :32], a[:, 32:]) * ds).sum()  # noqa: E731
        num[i] = (f(held + e) - f(held - e)) / 2e-5
    assert np.abs(f64(out) - num).max() < 1e-4   # (differences: h^2; the kernel: 2^-17 of terms of a few units)


def test_gate_far_and_infinite():
    gu = torch.zeros(4, 64, device="cuda")
    gu[0, :32], gu[0, 32:] = torch.linspace(-300, 300, 32), 1.0
    gu[1, :32], gu[1, 32:] = -3e38, 3e38
    gu[2, 3], gu[3, 40] = np.nan, np.inf
    codes, sf, ck, ck_sf = u8(4, 32), u8(4), u8(4, 64), u8(8)
    moe.moe_swiglu_mxfp8(gu, codes, sf, CANON, ckpt=ck, ckpt_sf=ck_sf)
    x = f64(gu)
    assert ref.mx8_close(codes[:1].cpu().numpy(), sf[:1].view(1, 1).cpu().numpy(), ref.swiglu(x[:1, :32], x[:1, 32:]), 2.0 ** -14)
    assert sf[1] == 0 and torch.all(codes[1] & 127 == 0) and sf[2] == 255 and sf[3] == 255
    assert ck_sf.tolist()[4:] == [255, 0, 0, 255]
    ds, out = torch.ones(4, 32, device="cuda"), torch.empty(4, 64, device="cuda")
    moe.moe_swiglu_mxfp8_backward(ds, ck, ck_sf, dgate_up=out)
    assert torch.isfinite(out[:2]).all() and torch.isnan(out[2, :32]).all()


# ------------------------------------------------------------------------------- the product

def mx_matrices(G, N, K, rng):
    """MXFP4 weights: packed codes [G, N, K / 2], tiled scales, values."""
    codes = rng.integers(0, 16, size=(G, N, K))
    sf = rng.integers(117, 123, size=(G, N, K // 32))
    packed = np.stack([ops_ref.pack(c) for c in codes])
    tiled = np.stack([ops_ref.tile_scales(s, fill=255) for s in sf])
    vals = np.stack([ops_ref.decode(c, s) for c, s in zip(codes, sf)])
    return torch.from_numpy(packed).cuda(), torch.from_numpy(tiled.reshape(-1)).cuda(), vals


def mx8_rows(cap, K, rng):
    x = rng.normal(size=(cap, K))
    c, s, v = ref.quant_mxfp8(x, True)
    return c.astype(np.uint8), s.astype(np.uint8), v


PRODUCTS = [  # N, K, rows of the groups
    (1, 128, [1]), (64, 128, [3, 0, 5]), (130, 256, [0, 0, 0]), (256, 384, [33, 1, 129]), (300, 128, [257, 0, 64, 300]),
    (96, 1024, [16, 17, 31, 32, 65]), (515, 640, [128, 512]), (257, 4096, [2]), (31, 256, [700]),
]


@pytest.mark.parametrize("N,K,counts", PRODUCTS)
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
def test_product(N, K, counts, out):
    rng = np.random.default_rng(N + K)
    G = len(counts)
    offsets = np.concatenate([[0], np.cumsum([(c + 127) // 128 * 128 for c in counts])])
    cap = max(int(offsets[-1]), 128)
    w, w_sf, wv = mx_matrices(G, N, K, rng)
    c, s, v = mx8_rows(cap, K, rng)
    dead = np.ones(cap, bool)
    for n, o in zip(counts, offsets):
        dead[o:o + n] = False
    c[dead], s[dead] = 127, 255
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = torch.full((cap, N + 3), -3.0, device="cuda").to(DT[out])
    d = lambda a: torch.from_numpy(np.asarray(a)).cuda()  # noqa: E731
    moe.moe_grouped_gemm_mxfp8(d(c), d(ops_ref.tile_scales(s)), d(np.int32(counts)), d(np.int32(offsets)), w, w_sf,
                               got[:, :N], status)
    assert status.item() == 0
    g64 = f64(got)
    assert np.all(g64[:, N:] == -3) and np.all(g64[dead] == -3)
    for g, (n, o) in enumerate(zip(counts, offsets)):
        ref_ = v[o:o + n] @ wv[g].T
        # products are exact; K roundings of 2^-24 of the sum of magnitudes at most
        slack = K * 2.0 ** -24 * (np.abs(v[o:o + n]) @ np.abs(wv[g]).T)
        assert np.all(ops_ref.rounded_ok(g64[o:o + n, :N], ref_, slack, out))


def test_product_of_all_rows_and_many_tiles():
    rng = np.random.default_rng(1)
    N, K, R = 700, 256, 1300
    w, w_sf, wv = mx_matrices(1, N, K, rng)
    c, s, v = mx8_rows(R, K, rng)
    out = torch.empty(R, N, device="cuda")
    d = lambda a: torch.from_numpy(np.asarray(a)).cuda()  # noqa: E731
    moe.moe_grouped_gemm_mxfp8(d(c), d(ops_ref.tile_scales(s)), None, None, w, w_sf, out)
    slack = K * 2.0 ** -24 * (np.abs(v) @ np.abs(wv[0]).T)
    assert np.all(np.abs(f64(out) - v @ wv[0].T) <= slack + 1e-30)
    again = torch.empty_like(out)
    moe.moe_grouped_gemm_mxfp8(d(c), d(ops_ref.tile_scales(s)), None, None, w, w_sf, again)
    assert torch.equal(out, again)


@pytest.mark.parametrize("G,most", [(1024, 300), (1024, 3), (619, 300), (618, 300)])
def test_product_of_many_groups(G, most):
    """Their starts leave the ring of stages less room (two stages of many rows, or four of few)."""
    rng = np.random.default_rng(G + most)
    N, K = 40, 640
    counts = rng.integers(0, 3, size=G)
    counts[[0, G // 2, G - 1]] = 0, most, 1
    offsets = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    cap = int(offsets[-1])
    w, w_sf, wv = mx_matrices(G, N, K, rng)
    c, s, v = (np.zeros(z) for z in ((cap, K), (cap, K // 32), (cap, K)))
    live = np.concatenate([np.arange(o, o + n) for n, o in zip(counts, offsets)])
    c[live], s[live], v[live] = mx8_rows(len(live), K, rng)
    c, s = c.astype(np.uint8), s.astype(np.uint8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = torch.full((cap, N), -3.0, device="cuda")
    d = lambda a: torch.from_numpy(np.asarray(a)).cuda()  # noqa: E731
    moe.moe_grouped_gemm_mxfp8(d(c), d(ops_ref.tile_scales(s)), d(np.int32(counts)), d(np.int32(offsets)), w, w_sf,
                               got, status)
    assert status.item() == 0
    g64 = f64(got)
    dead = np.ones(cap, bool)
    dead[live] = False
    assert np.all(g64[dead] == -3)
    for g, (n, o) in enumerate(zip(counts, offsets)):
        slack = K * 2.0 ** -24 * (np.abs(v[o:o + n]) @ np.abs(wv[g]).T)
        assert np.all(np.abs(g64[o:o + n] - v[o:o + n] @ wv[g].T) <= slack)


def test_product_scales_of_every_block():
    """Rows and weights of ones, block scales of their own: every scale meets its block."""
    N, K, R = 140, 512, 150
    rng = np.random.default_rng(2)
    sa, sw = rng.integers(120, 134, size=(R, K // 32)), rng.integers(120, 134, size=(N, K // 32))
    a = torch.full((R, K), 0x38, dtype=torch.uint8, device="cuda")           # 1.0
    w = torch.full((1, N, K // 2), 0x22, dtype=torch.uint8, device="cuda")   # 1.0, 1.0
    out = torch.empty(R, N, device="cuda")
    d = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    moe.moe_grouped_gemm_mxfp8(a, d(ops_ref.tile_scales(sa)), None, None, w, d(ops_ref.tile_scales(sw)), out)
    want = 32 * (2.0 ** (sa - 127.0)) @ (2.0 ** (sw - 127.0)).T
    # K / 32 = 16 MMAs, each of 32 equal powers of two, spread over 26 binary places: each truncates the sum
    # it leaves (of positive numbers) by at most a unit of the last of 24 places
    assert np.all(np.abs(f64(out) - want) <= 16 * 2.0 ** -23 * want)


def test_product_of_nan_and_largest():
    N, K, R = 32, 128, 4
    a = torch.full((R, K), 0x7E, dtype=torch.uint8, device="cuda")           # 448
    a[1, 5], a[2, 6] = 0x7F, 0xFE                                            # NaN, -448
    sf = np.full((R, 4), 127)
    sf[3, 2] = 255
    w = torch.full((1, N, K // 2), 0x77, dtype=torch.uint8, device="cuda")   # 6.0
    out = torch.empty(R, N, device="cuda")
    d = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    moe.moe_grouped_gemm_mxfp8(a, d(ops_ref.tile_scales(sf)), None, None, w,
                               d(ops_ref.tile_scales(np.full((N, 4), 127))), out)
    assert torch.all(out[0] == 448 * 6 * 128) and torch.isnan(out[1]).all()
    assert torch.all(out[2] == 448 * 6 * 126) and torch.isnan(out[3]).all()


def test_bad_groups_are_skipped():
    rng = np.random.default_rng(3)
    w, w_sf, _ = mx_matrices(3, 64, 128, rng)
    c, s, v = mx8_rows(384, 128, rng)
    out = torch.full((384, 64), -3.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = lambda a: torch.from_numpy(np.asarray(a)).cuda()  # noqa: E731
    moe.moe_grouped_gemm_mxfp8(d(c), d(ops_ref.tile_scales(s)), d(np.int32([5, 9, 200])), d(np.int32([0, 130, 256, 384])),
                               w, w_sf, out, status)
    assert status.item() == moe.MOE_DEV_BAD_INDEX
    assert torch.all(out[5:] == -3) and not torch.any(out[:5] == -3)
