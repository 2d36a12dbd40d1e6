"""The operators around the experts on tensors of over 2^31 elements: the last rows are what a call on
those rows alone gives; and calls on streams and in graphs of their own."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu
CANON, TILED = moe.MOE_SF_CANONICAL, moe.MOE_SF_TILED


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device="cuda")


@pytest.fixture(autouse=True)
def room():
    yield
    torch.cuda.empty_cache()


def filled(rows, cols, last):
    """bf16 rows of which the last few are random, the others ones."""
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-last:] = torch.randn(last, cols, device="cuda").bfloat16()
    return x


def test_norm_and_its_gradient():
    T, H, n = 132000, 16384, 5
    x, w = filled(T, H, n), torch.rand(H, device="cuda").bfloat16()
    y, codes, sf, rstd = torch.empty_like(x), u8(T, H), u8(T * H // 32), torch.empty(T, device="cuda")
    moe.moe_rmsnorm(x, w, 1e-6, y=y, codes=codes, sf=sf, sf_layout=CANON, rstd=rstd)
    y2, c2, s2, r2 = torch.empty(n, H, device="cuda").bfloat16(), u8(n, H), u8(n * H // 32), torch.empty(n, device="cuda")
    moe.moe_rmsnorm(x[-n:], w, 1e-6, y=y2, codes=c2, sf=s2, sf_layout=CANON, rstd=r2)
    assert torch.equal(y[-n:], y2) and torch.equal(codes[-n:], c2) and torch.equal(sf[-n * H // 32:], s2)
    assert torch.equal(rstd[-n:], r2) and torch.equal(y[0], y[T // 2])
    del codes, sf
    dx, dx2 = torch.empty_like(x), torch.empty_like(y2)
    moe.moe_rmsnorm_backward(y, x, w, rstd, dx)
    moe.moe_rmsnorm_backward(y[-n:], x[-n:], w, r2, dx2)
    assert torch.equal(dx[-n:], dx2) and torch.equal(dx[0], dx[T // 2])


def test_quantiser():
    R, C, n = 263000, 16384, 4
    x = filled(R, C, n)
    codes, sf = u8(R, C), u8(moe.moe_mxfp4_scale_bytes(1, R, C, TILED))
    moe.moe_quant_mxfp8(x, codes, sf, TILED)
    c2, s2 = u8(n, C), u8(n * C // 32)
    moe.moe_quant_mxfp8(x[-n:], c2, s2, CANON)
    assert torch.equal(codes[-n:], c2) and torch.all(codes[R // 2] == codes[0, 0])
    r = torch.arange(R - n, R, device="cuda")[:, None]
    b = torch.arange(C // 32, device="cuda")[None, :]
    at = ((r >> 7) * (C // 128) + (b >> 2)) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    assert torch.equal(sf[at].view(-1), s2)


def test_gate_and_its_gradient():
    R, I, n = 140000, 8192, 3
    gu = filled(R, 2 * I, n)
    codes, sf, ck, ck_sf = u8(R, I), u8(R * I // 32), u8(R, 2 * I), u8(R * I // 16)
    moe.moe_swiglu_mxfp8(gu, codes, sf, CANON, ckpt=ck, ckpt_sf=ck_sf)
    c2, s2, k2, ks2 = u8(n, I), u8(n * I // 32), u8(n, 2 * I), u8(n * I // 16)
    moe.moe_swiglu_mxfp8(gu[-n:], c2, s2, CANON, ckpt=k2, ckpt_sf=ks2)
    assert torch.equal(codes[-n:], c2) and torch.equal(sf[-n * I // 32:], s2)
    assert torch.equal(ck[-n:], k2) and torch.equal(ck_sf[-n * I // 16:], ks2)
    del codes, sf
    ds = gu[:, :I]
    d, d_sf, dgu = u8(R, 2 * I), u8(R * I // 16), torch.empty_like(gu)
    moe.moe_swiglu_mxfp8_backward(ds, ck, ck_sf, d, d_sf, CANON, dgate_up=dgu)
    d2, ds2, dgu2 = u8(n, 2 * I), u8(n * I // 16), torch.empty_like(gu[-n:])
    moe.moe_swiglu_mxfp8_backward(ds[-n:], k2, ks2, d2, ds2, CANON, dgate_up=dgu2)
    assert torch.equal(d[-n:], d2) and torch.equal(d_sf[-n * I // 16:], ds2) and torch.equal(dgu[-n:], dgu2)
    assert torch.equal(dgu[0], dgu[R // 2])


def test_routing_and_its_gradient():
    T, E, k, n = 6_800_000, 320, 4, 7
    l = torch.zeros(T, E, device="cuda")
    l[:, 5], l[:, 300] = 2.0, 3.0
    l[-n:] = torch.randn(n, E, device="cuda")
    bias = torch.rand(E, device="cuda") * 0.1
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    how = dict(score=moe.MOE_SCORE_SIGMOID)
    moe.moe_route_scores(l, ids, w, bias=bias, num_groups=8, topk_groups=8, **how)
    i2, w2 = torch.empty(n, k, dtype=torch.int32, device="cuda"), torch.empty(n, k, device="cuda")
    moe.moe_route_scores(l[-n:], i2, w2, bias=bias, num_groups=8, topk_groups=8, **how)
    assert torch.equal(ids[-n:], i2) and torch.equal(w[-n:], w2)
    assert ids[T // 2, :2].tolist() == [300, 5] and torch.equal(ids[0], ids[T // 2])
    dl, d2 = torch.empty_like(l), torch.empty(n, E, device="cuda")
    moe.moe_route_scores_backward(l, ids, w, dl, **how)
    moe.moe_route_scores_backward(l[-n:], i2, w2, d2, **how)
    assert torch.equal(dl[-n:], d2) and torch.equal(dl[0], dl[T // 2])


def test_product():
    R, N, K, n = 531000, 32, 4096, 130
    R = R // 128 * 128 + n            # the last block of rows begins on a multiple of 128
    a = torch.full((R, K), 0x38, dtype=torch.uint8, device="cuda")
    a[-n:] = torch.randint(0, 120, (n, K), dtype=torch.uint8, device="cuda")
    sf = torch.full((moe.moe_mxfp4_scale_bytes(1, R, K, TILED),), 127, dtype=torch.uint8, device="cuda")
    w = torch.randint(0, 256, (1, N, K // 2), dtype=torch.uint8, device="cuda")
    w_sf = torch.full((moe.moe_mxfp4_scale_bytes(1, N, K, TILED),), 120, dtype=torch.uint8, device="cuda")
    out, last = torch.empty(R, N, device="cuda"), torch.empty(n, N, device="cuda")
    moe.moe_grouped_gemm_mxfp8(a, sf, None, None, w, w_sf, out)
    moe.moe_grouped_gemm_mxfp8(a[-n:], sf[:moe.moe_mxfp4_scale_bytes(1, n, K, TILED)], None, None, w, w_sf, last)
    assert torch.equal(out[-n:], last) and torch.equal(out[0], out[R // 2])


def test_two_streams_at_once_and_a_graph_on_a_third():
    """The same calls on buffers of their own, on two streams at a time and captured on another."""
    T, H, I = 300, 256, 128
    g = torch.Generator("cuda").manual_seed(0)
    w = torch.randint(0, 256, (1, 2 * I, H // 2), dtype=torch.uint8, device="cuda", generator=g)
    w_sf = torch.full((moe.moe_mxfp4_scale_bytes(1, 2 * I, H, TILED),), 120, dtype=torch.uint8, device="cuda")

    def state(seed):
        g = torch.Generator("cuda").manual_seed(seed)
        return dict(x=torch.randn(T, H, generator=g, device="cuda").bfloat16(), codes=u8(T, H),
                    sf=u8(moe.moe_mxfp4_scale_bytes(1, T, H, TILED)), gu=torch.empty(T, 2 * I, device="cuda"),
                    s=u8(T, I), s_sf=u8(moe.moe_mxfp4_scale_bytes(1, T, I, TILED)), ck=u8(T, 2 * I),
                    ck_sf=u8(T * I // 16), ds=torch.randn(T, I, generator=g, device="cuda"),
                    d=torch.empty(T, 2 * I, device="cuda"))

    def step(s):
        moe.moe_rmsnorm(s["x"], None, 1e-6, codes=s["codes"], sf=s["sf"])
        moe.moe_grouped_gemm_mxfp8(s["codes"], s["sf"], None, None, w, w_sf, s["gu"])
        moe.moe_swiglu_mxfp8(s["gu"], s["s"], s["s_sf"], TILED, ckpt=s["ck"], ckpt_sf=s["ck_sf"])
        moe.moe_swiglu_mxfp8_backward(s["ds"], s["ck"], s["ck_sf"], dgate_up=s["d"])

    states = [state(i) for i in range(3)]
    want = []
    for s in states:
        step(s)
        want.append((s["s"].clone(), s["d"].clone()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(states[2])
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in states:
        s["s"].zero_(), s["d"].zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for st, s in zip(streams, states[:2]):
            with torch.cuda.stream(st):
                step(s)
        with torch.cuda.stream(streams[2]):
            graph.replay()
    torch.cuda.synchronize()
    for s, (a, b) in zip(states, want):
        assert torch.equal(s["s"], a) and torch.equal(s["d"], b)
