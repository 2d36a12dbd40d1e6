"""The root-mean-square norm with the residual's addition and its 8-bit result, and its gradient, against
64-bit implementations."""
import numpy as np
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
import ops8_ref as ref
import ops_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
# The mean square is a sum of positive terms of which a thread adds up at most 16 and ten additions join
# them: 27 roundings, half of that in its root; rsqrt is within 2 ulp (2^-22); two products more.
Y_TOL = 14 * 2.0 ** -24 + 2.0 ** -22 + 2 * 2.0 ** -24
SIZES = [(1, 1), (3, 8), (2, 31), (5, 32), (300, 64), (7, 96), (65, 250), (129, 256), (4, 260), (33, 512),
         (3, 520), (40, 1001), (6, 2048), (700, 2056), (3, 4096), (2, 4100), (2, 8192), (1, 16384),
         (3, 16383)]


def rows(T, H, dtype, g, pad=0, off=0, scale=1.0):
    """[T, H] rows of H + pad elements that start off elements into a buffer."""
    buf = torch.randn(T * (H + pad) + off + 8, generator=g, device="cuda").mul_(scale).to(DT[dtype])
    return buf[off:off + T * (H + pad)].view(T, H + pad)[:, :H]


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 8), (3, 1)])
def test_norm(T, H, dtype, pad, off):
    g = torch.Generator("cuda").manual_seed(H)
    x, r = rows(T, H, dtype, g, pad, off, 3.0), rows(T, H, dtype, g, pad, off)
    w = rows(1, H, dtype, g)[0]
    for res in (None, r):
        h = torch.full((T, H + pad), 5.0, device="cuda").to(DT[dtype])[:, :H] if res is not None else None
        y, rstd = rows(T, H, dtype, g, pad, off), torch.empty(T, device="cuda")
        edge = y.as_strided((T, pad), (H + pad, 1), y.storage_offset() + H).clone()
        q = H % 32 == 0
        codes = torch.zeros(T, H, dtype=torch.uint8, device="cuda") if q else None
        for layout in (moe.MOE_SF_CANONICAL, moe.MOE_SF_TILED):
            n = moe.moe_mxfp4_scale_bytes(1, T, H, layout) if q else 0
            sf = torch.full((n,), 77, dtype=torch.uint8, device="cuda") if q else None
            for rule in (moe.MOE_MX_CEIL, moe.MOE_MX_FLOOR):
                moe.moe_rmsnorm(x, w, EPS, residual=res, h=h, y=y, rstd=rstd, codes=codes, sf=sf,
                                sf_layout=layout, scale_rule=rule)
                sum_ = x if res is None else (x.float() + r.float()).to(DT[dtype])
                if res is not None:
                    assert torch.equal(h, sum_)
                want, want_rstd = ref.rmsnorm(f64(sum_), f64(w), EPS)
                assert np.all(np.abs(f64(rstd) - want_rstd) <= Y_TOL * want_rstd)
                assert np.all(ops_ref.rounded_ok(f64(y), want, Y_TOL * np.abs(want), dtype))
                assert torch.equal(edge, y.as_strided((T, pad), (H + pad, 1), y.storage_offset() + H))
                if q:
                    s = sf.cpu().numpy()
                    s = s.reshape(T, H // 32) if layout == moe.MOE_SF_CANONICAL else ref.untile(s, T, H // 32)
                    assert ref.mx8_close(codes.cpu().numpy(), s, want, Y_TOL, rule == moe.MOE_MX_CEIL)
                    if layout == moe.MOE_SF_TILED and (H // 32) % 4:  # blocks past the row's end
                        t = ref.untile(sf.cpu().numpy(), T, (H // 32 + 3) // 4 * 4)
                        assert np.all(t[:, H // 32:] == 0)
            if not q:
                break


def test_weight_of_ones_and_single_outputs():
    x = torch.randn(9, 320, device="cuda").bfloat16()
    ones = torch.ones(320, device="cuda").bfloat16()
    a, b, c = (torch.empty_like(x) for _ in range(3))
    moe.moe_rmsnorm(x, ones, EPS, y=a)
    moe.moe_rmsnorm(x, None, EPS, y=b)
    assert torch.equal(a, b)
    rstd = torch.empty(9, device="cuda")
    moe.moe_rmsnorm(x, None, EPS, rstd=rstd)
    codes, sf = torch.empty(9, 320, dtype=torch.uint8, device="cuda"), torch.empty(90, dtype=torch.uint8, device="cuda")
    moe.moe_rmsnorm(x, ones, EPS, codes=codes, sf=sf, sf_layout=moe.MOE_SF_CANONICAL)
    want, want_rstd = ref.rmsnorm(f64(x), 1.0, EPS)
    assert np.all(np.abs(f64(rstd) - want_rstd) <= Y_TOL * want_rstd)
    assert ref.mx8_close(codes.cpu().numpy(), sf.cpu().numpy().reshape(9, 10), want, Y_TOL)
    moe.moe_rmsnorm(x, ones, EPS, residual=a, h=c)
    assert torch.equal(c, (x.float() + a.float()).bfloat16())


@pytest.mark.parametrize("H", [64, 1000, 4096])
def test_in_place(H):
    g = torch.Generator("cuda").manual_seed(1)
    x, r, w = rows(50, H, "bf16", g), rows(50, H, "bf16", g), rows(1, H, "bf16", g)[0]
    h, y = torch.empty_like(x), torch.empty_like(x)
    moe.moe_rmsnorm(x, w, EPS, residual=r, h=h, y=y)
    for into in ("residual", "x"):
        x2, r2 = x.clone(), r.clone()
        if into == "residual":
            moe.moe_rmsnorm(x2, w, EPS, residual=r2, h=r2, y=x2)
            assert torch.equal(r2, h) and torch.equal(x2, y)
        else:
            y2 = torch.empty_like(x)
            moe.moe_rmsnorm(x2, w, EPS, residual=r2, h=x2, y=y2)
            assert torch.equal(x2, h) and torch.equal(y2, y) and torch.equal(r2, r)


def test_zero_and_infinite_rows():
    x = torch.randn(5, 64, device="cuda")
    x[1], x[2, 5], x[3, 7] = 0, np.inf, np.nan
    x[4] = torch.finfo(torch.float32).max     # the square is past 32 bits
    y, codes = torch.empty_like(x), torch.full((5, 64), 9, dtype=torch.uint8, device="cuda")
    sf = torch.empty(10, dtype=torch.uint8, device="cuda")
    moe.moe_rmsnorm(x, None, EPS, y=y, codes=codes, sf=sf, sf_layout=moe.MOE_SF_CANONICAL)
    sf = sf.view(5, 2)
    assert torch.isfinite(y[0]).all() and torch.all(y[1] == 0) and torch.isnan(y[3]).all()
    assert torch.isnan(y[2, 5]) and torch.all(y[2, :5] == 0) and torch.all(y[4] == 0)
    assert torch.all(sf[1] == 0) and torch.all(codes[1] == 0)
    assert sf[2, 0] == 255 and torch.all(sf[3] == 255) and torch.all(codes[3] == 0)
    # a row of NaN changes no other row
    z = torch.empty_like(y)
    moe.moe_rmsnorm(x[:1], None, EPS, y=z[:1])
    assert torch.equal(y[0], z[0])


@pytest.mark.parametrize("T,H", SIZES + [(3000, 64), (5000, 40)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1)])
def test_gradient(T, H, dtype, pad, off):
    g = torch.Generator("cuda").manual_seed(H + 1)
    dy, h, dh = (rows(T, H, dtype, g, pad, off) for _ in range(3))
    w = rows(1, H, dtype, g)[0]
    rstd = torch.from_numpy(1 / np.sqrt((f64(h) ** 2).mean(1) + EPS)).float().cuda()
    ws = torch.empty(moe.moe_rmsnorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    for extra in (None, dh):
        for weight in (w, None):
            dx, dw = rows(T, H, dtype, g, pad, off), torch.full((H,), -3.0, device="cuda")
            moe.moe_rmsnorm_backward(dy, h, weight, rstd, dx, dw, ws, dh=extra)
            wf = f64(w) if weight is not None else np.ones(H)
            d64, h64, r64 = f64(dy), f64(h), f64(rstd)
            e64 = f64(dh) if extra is not None else np.zeros((T, H))
            want, want_w = ref.rmsnorm_grad(d64, h64, wf, r64, e64)
            # the row's sum: at most 27 roundings of terms |dy w x^|, then a few of each term
            x = np.abs(h64 * r64[:, None])
            mean = (np.abs(d64 * wf) * x).mean(1, keepdims=True)
            slack = r64[:, None] * (4 * 2.0 ** -24 * np.abs(d64 * wf) + 36 * 2.0 ** -24 * x * mean)
            slack = slack + 2.0 ** -23 * (np.abs(e64) + r64[:, None] * (np.abs(d64 * wf) + x * mean))
            assert np.all(ops_ref.rounded_ok(f64(dx), want, slack, dtype))
            # the rows of a part (at least 152 parts with their share of the rows, or as many as the
            # workspace holds), short rows' eight warps, then the parts by 32 threads
            most = max(1, moe.moe_rmsnorm_workspace_size(T, H) // (4 * H))
            n = -(-T // 152) + 8 + -(-most // 32) + 5 + 2
            assert np.all(np.abs(f64(dw) - want_w) <= n * 2.0 ** -24 * (np.abs(d64) * x).sum(0) + 1e-37)
            again = torch.empty_like(dw)
            moe.moe_rmsnorm_backward(dy, h, weight, rstd, dx, again, ws, dh=extra)
            assert torch.equal(dw, again)
    alone = torch.empty(T, H, device="cuda").to(DT[dtype])
    moe.moe_rmsnorm_backward(dy, h, None, rstd, alone, dh=dh)
    assert torch.equal(alone, dx)


def test_gradient_against_differences():
    rng = np.random.default_rng(0)
    T, H = 3, 24
    x, w, dy, dh = rng.normal(size=(T, H)), rng.normal(size=H), rng.normal(size=(T, H)), rng.normal(size=(T, H))
    x, w, dy, dh = (a.astype(np.float32).astype(np.float64) for a in (x, w, dy, dh))

    def loss(a, b):
        return (ref.rmsnorm(a, b, EPS)[0] * dy).sum() + (a * dh).sum()

    d = lambda a: torch.from_numpy(a).float().cuda()  # noqa: E731
    dx, dw, rstd = torch.empty(T, H, device="cuda"), torch.empty(H, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_rmsnorm(d(x), d(w), EPS, rstd=rstd)
    ws = torch.empty(moe.moe_rmsnorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    moe.moe_rmsnorm_backward(d(dy), d(x), d(w), rstd, dx, dw, ws, dh=d(dh))
    for a, got in ((x, dx), (w, dw)):
        num = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            e = np.zeros_like(a)
            e[i] = 1e-5
            f = (lambda s: loss(x + s, w)) if a is x else (lambda s: loss(x, w + s))
            num[i] = (f(e) - f(-e)) / 2e-5
        # differences are off by h^2 times a third derivative and 2^-53 / h; the kernel by some 2^-20
        assert np.abs(f64(got) - num).max() < 1e-4


def test_gradient_in_place():
    g = torch.Generator("cuda").manual_seed(9)
    dy, h, dh = (rows(40, 1024, "bf16", g) for _ in range(3))
    rstd = torch.rand(40, device="cuda") + 0.5
    want = torch.empty_like(dy)
    moe.moe_rmsnorm_backward(dy, h, None, rstd, want, dh=dh)
    for name in ("dy", "dh", "h"):
        t = dict(dy=dy.clone(), dh=dh.clone(), h=h.clone())
        moe.moe_rmsnorm_backward(t["dy"], t["h"], None, rstd, t[name], dh=t["dh"])
        assert torch.equal(t[name], want)


def test_no_rows():
    x, dw = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    moe.moe_rmsnorm(x, None, EPS, y=x)
    moe.moe_rmsnorm_backward(x, x, None, torch.empty(0, device="cuda"), x, dw)
    assert torch.all(dw == 0)


def test_in_a_graph_and_on_another_stream():
    T, H = 600, 512
    x, r, w = torch.randn(T, H, device="cuda"), torch.randn(T, H, device="cuda"), torch.randn(H, device="cuda")
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    ws = torch.empty(moe.moe_rmsnorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        moe.moe_rmsnorm(x, w, EPS, residual=r, h=h, y=y, rstd=rstd, stream=stream)
        moe.moe_rmsnorm_backward(y, h, w, rstd, dx, dw, ws, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(torch.randn_like(x))
    step()
    want = [t.clone() for t in (h, y, dx, dw)]
    for t in (h, y, dx, dw):
        t.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip((h, y, dx, dw), want))
    for t in (h, y, dx, dw):
        t.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((h, y, dx, dw), want))
