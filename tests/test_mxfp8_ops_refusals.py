"""Argument checks of the operators around the experts: the library's own, answered on the host before
any launch (the pointers given here are never read), and the binding's."""
import ctypes as C

import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
from nvfp4_mixture_experts_gb300 import build as moe_build
from stand_in import CPU, install

P = C.c_void_p(4096)      # a well aligned address that nothing reads
ODD = C.c_void_p(4104)    # a multiple of 8 alone
HALF = C.c_void_p(4098)   # of 2
BYTE = C.c_void_p(4097)
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


def call(lib, name, defaults, **kw):
    args = dict(defaults)
    assert set(kw) <= set(args), kw
    args.update(kw)
    return getattr(lib, name)(*args.values())


ROUTE = dict(l=P, dtype=0, stride=64, bias=None, T=4, E=64, k=4, score=0, groups=1, topg=1, gs=0, renorm=1,
             scale=1.0, ids=P, w=P, stream=None)
ROUTE_BACK = dict(l=P, dtype=0, stride=64, ids=P, dw=P, T=4, E=64, k=4, score=0, renorm=1, scale=1.0, dl=P,
                  dstride=64, stream=None)
NORM = dict(x=P, dtype=0, xs=64, r=P, rs=64, w=P, eps=1e-6, T=4, H=64, h=P, hs=64, y=P, ys=64, rstd=P, codes=P,
            sf=P, layout=1, rule=1, stream=None)
NORM_BACK = dict(dy=P, dtype=0, dys=1024, dh=P, dhs=1024, h=P, hs=1024, w=P, rstd=P, T=4, H=1024, dx=P, dxs=1024,
                 dw=P, ws=P, ws_bytes=4 * 1024 * 4, stream=None)
QUANT = dict(x=P, dtype=0, batch=1, rows=4, cols=64, rs=64, bs=0, rule=0, perm=None, codes=P, sf=P, layout=1,
             values=None, stream=None)
GATE = dict(gu=P, dtype=0, stride=128, rows=4, inter=64, perm=None, rule=1, codes=P, sf=P, layout=1, ck=P,
            ck_sf=P, stream=None)
GATE_BACK = dict(ds=P, dtype=0, stride=64, ck=P, ck_sf=P, rows=4, inter=64, perm=None, rule=1, codes=P, sf=P,
                 layout=1, dgu=P, stream=None)
GEMM = dict(a=P, a_sf=P, cap=128, counts=P, offsets=P, G=2, w=P, w_sf=P, N=64, K=128, out=P, dtype=0, stride=64,
            status=None, stream=None)

INVALID = [
    ("moe_route_scores", ROUTE, [
        dict(dtype=3), dict(T=-1), dict(E=0), dict(k=0), dict(k=65), dict(score=2), dict(score=-1), dict(groups=0),
        dict(groups=7), dict(groups=4, topg=0), dict(groups=4, topg=5), dict(groups=32, topg=1), dict(gs=2),
        dict(renorm=2), dict(l=None), dict(ids=None), dict(w=None), dict(stride=63), dict(l=BYTE),
        dict(l=HALF, dtype=2), dict(bias=HALF), dict(ids=HALF), dict(w=HALF)]),
    ("moe_route_scores_backward", ROUTE_BACK, [
        dict(dtype=-1), dict(T=-1), dict(E=0), dict(k=0), dict(k=65), dict(score=2), dict(renorm=-1), dict(l=None),
        dict(ids=None), dict(dw=None), dict(dl=None), dict(stride=63), dict(dstride=63), dict(l=BYTE), dict(dl=BYTE),
        dict(ids=HALF), dict(dw=HALF), dict(dl=HALF, dtype=2)]),
    ("moe_rmsnorm", NORM, [
        dict(dtype=3), dict(T=-1), dict(H=0), dict(eps=-1.0), dict(eps=float("nan")), dict(r=None), dict(x=None),
        dict(codes=None), dict(sf=None), dict(layout=2), dict(rule=2), dict(xs=63), dict(rs=63), dict(hs=63),
        dict(ys=63), dict(x=BYTE), dict(r=BYTE), dict(w=BYTE), dict(h=BYTE), dict(y=BYTE), dict(rstd=HALF),
        dict(codes=ODD), dict(sf=ODD), dict(h=None, y=None, rstd=None, codes=None, sf=None)]),
    ("moe_rmsnorm_backward", NORM_BACK, [
        dict(dtype=3), dict(T=-1), dict(H=0), dict(dy=None), dict(h=None), dict(rstd=None), dict(dx=None),
        dict(dys=1023), dict(hs=1023), dict(dxs=1023), dict(dhs=1023), dict(dy=BYTE), dict(dh=BYTE), dict(h=BYTE),
        dict(w=BYTE), dict(dx=BYTE), dict(dw=HALF), dict(rstd=HALF), dict(ws=None), dict(ws=ODD)]),
    ("moe_quant_mxfp8", QUANT, [
        dict(dtype=3), dict(batch=-1), dict(rows=-1), dict(cols=0), dict(rule=2), dict(layout=2), dict(x=None),
        dict(codes=None), dict(sf=None), dict(rs=63), dict(codes=ODD), dict(values=ODD), dict(x=BYTE), dict(sf=ODD),
        dict(perm=P, batch=2), dict(perm=HALF)]),
    ("moe_swiglu_mxfp8", GATE, [
        dict(dtype=3), dict(rows=-1), dict(inter=0), dict(layout=2), dict(rule=-1), dict(gu=None), dict(codes=None),
        dict(sf=None), dict(ck=None), dict(ck_sf=None), dict(stride=127), dict(gu=BYTE), dict(perm=HALF),
        dict(codes=ODD), dict(sf=ODD), dict(ck=ODD)]),
    ("moe_swiglu_mxfp8_backward", GATE_BACK, [
        dict(dtype=3), dict(rows=-1), dict(inter=0), dict(layout=2), dict(rule=2), dict(ds=None), dict(ck=None),
        dict(ck_sf=None), dict(codes=None), dict(sf=None), dict(codes=None, sf=None, dgu=None), dict(stride=63),
        dict(ds=BYTE), dict(perm=HALF), dict(codes=ODD), dict(sf=ODD), dict(ck=ODD), dict(dgu=ODD)]),
    ("moe_grouped_gemm_mxfp8", GEMM, [
        dict(dtype=3), dict(cap=-1), dict(G=0), dict(N=0), dict(K=0), dict(counts=None), dict(offsets=None),
        dict(counts=None, offsets=None), dict(a=None), dict(a_sf=None), dict(w=None), dict(w_sf=None),
        dict(out=None), dict(stride=63), dict(a=ODD), dict(a_sf=ODD), dict(w=ODD), dict(w=C.c_void_p(4112)),
        dict(w_sf=ODD), dict(out=BYTE), dict(status=HALF)]),
]
UNSUPPORTED = [
    ("moe_route_scores", ROUTE, [dict(E=1025, stride=1025), dict(k=33), dict(groups=64, topg=4)]),
    ("moe_route_scores_backward", ROUTE_BACK, [dict(E=1025, stride=1025, dstride=1025), dict(k=33)]),
    ("moe_rmsnorm", NORM, [dict(H=16385, xs=BIG, rs=BIG, hs=BIG, ys=BIG), dict(H=48)]),
    ("moe_rmsnorm_backward", NORM_BACK, [dict(H=16385)]),
    ("moe_quant_mxfp8", QUANT, [dict(cols=48, rs=48), dict(batch=BIG, rows=BIG)]),
    ("moe_swiglu_mxfp8", GATE, [dict(inter=48), dict(inter=2 ** 28 + 32), dict(rows=BIG)]),
    ("moe_swiglu_mxfp8_backward", GATE_BACK, [dict(inter=48), dict(rows=BIG)]),
    ("moe_grouped_gemm_mxfp8", GEMM, [dict(K=96), dict(K=64), dict(G=1025), dict(G=1024, N=2 ** 22)]),
]
NOTHING = [  # nothing to do: no pointer is needed
    ("moe_route_scores", ROUTE, dict(T=0, l=None, ids=None, w=None)),
    ("moe_route_scores_backward", ROUTE_BACK, dict(T=0, l=None, ids=None, dw=None, dl=None)),
    ("moe_rmsnorm", NORM, dict(T=0, x=None, r=None, h=None, y=None, rstd=None, codes=None, sf=None)),
    ("moe_rmsnorm_backward", NORM_BACK, dict(T=0, dy=None, h=None, rstd=None, dx=None, dw=None, ws=None, ws_bytes=0)),
    ("moe_quant_mxfp8", QUANT, dict(rows=0, x=None, codes=None, sf=None)),
    ("moe_swiglu_mxfp8", GATE, dict(rows=0, gu=None, codes=None, sf=None, ck=None, ck_sf=None)),
    ("moe_swiglu_mxfp8_backward", GATE_BACK, dict(rows=0, ds=None, ck=None, ck_sf=None, codes=None, sf=None, dgu=None)),
    ("moe_grouped_gemm_mxfp8", GEMM, dict(cap=0, a=None, a_sf=None, out=None)),
]


@pytest.mark.parametrize("name,defaults,cases", INVALID, ids=[c[0] for c in INVALID])
def test_invalid_arguments(lib, name, defaults, cases):
    for kw in cases:
        assert call(lib, name, defaults, **kw) == moe.MOE_ERR_INVALID, kw


@pytest.mark.parametrize("name,defaults,cases", UNSUPPORTED, ids=[c[0] for c in UNSUPPORTED])
def test_unsupported_arguments(lib, name, defaults, cases):
    for kw in cases:
        assert call(lib, name, defaults, **kw) == moe.MOE_ERR_UNSUPPORTED, kw


@pytest.mark.parametrize("name,defaults,kw", NOTHING, ids=[c[0] for c in NOTHING])
def test_nothing_to_do(lib, name, defaults, kw):
    assert call(lib, name, defaults, **kw) == moe.MOE_OK


def test_a_workspace_that_is_too_small(lib):
    assert call(lib, "moe_rmsnorm_backward", NORM_BACK, ws_bytes=0, ws=None) == moe.MOE_ERR_WORKSPACE
    assert call(lib, "moe_rmsnorm_backward", NORM_BACK, ws_bytes=4 * 1024 * 4 - 1) == moe.MOE_ERR_WORKSPACE


def test_workspace_sizes():
    size = moe.moe_rmsnorm_workspace_size
    assert size(1, 64) == 0 and size(0, 64) == 0 and size(-1, 64) == 0 and size(4, 0) == 0 and size(4, 16385) == 0
    assert size(4, 1024) == 4 * 1024 * 4 and size(8, 64) == 0 and size(9, 64) == 2 * 64 * 4
    for T in (9, 1000, 10 ** 6, BIG):
        for H in (1, 512, 513, 4096, 16384):
            assert 0 < size(T, H) <= 32 << 20


# ------------------------------------------------------------------------------- the binding

def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def f32(*shape):
    return torch.zeros(*shape)


def calls():
    """name -> (function, arguments that fit)."""
    T, E, k, H, R, I, G, N, K = 4, 64, 3, 96, 5, 64, 3, 32, 128
    c = moe.MOE_SF_CANONICAL
    return {
        "moe_route_scores": (moe.moe_route_scores, dict(logits=f32(T, E), topk_ids=i32(T, k), topk_w=f32(T, k), bias=f32(E))),
        "moe_route_scores_backward": (moe.moe_route_scores_backward, dict(
            logits=f32(T, E), topk_ids=i32(T, k), dtopk_w=f32(T, k), dlogits=f32(T, E))),
        "moe_rmsnorm": (moe.moe_rmsnorm, dict(
            x=f32(T, H), weight=f32(H), eps=1e-6, residual=f32(T, H), h=f32(T, H), y=f32(T, H), rstd=f32(T),
            codes=u8(T, H), sf=u8(T * H // 32), sf_layout=c)),
        "moe_rmsnorm_backward": (moe.moe_rmsnorm_backward, dict(
            dy=f32(T, H), h=f32(T, H), weight=f32(H), rstd=f32(T), dx=f32(T, H), dweight=f32(H), ws=u8(T * H * 4),
            dh=f32(T, H))),
        "moe_quant_mxfp8": (moe.moe_quant_mxfp8, dict(
            x=f32(R, H), codes=u8(R, H), sf=u8(R * H // 32), sf_layout=c, perm_src=i32(R), values=f32(R, H))),
        "moe_swiglu_mxfp8": (moe.moe_swiglu_mxfp8, dict(
            gate_up=f32(R, 2 * I), codes=u8(R, I), sf=u8(R * I // 32), sf_layout=c, ckpt=u8(R, 2 * I),
            ckpt_sf=u8(R * I // 16), perm_src=i32(R))),
        "moe_swiglu_mxfp8_backward": (moe.moe_swiglu_mxfp8_backward, dict(
            ds=f32(R, I), ckpt=u8(R, 2 * I), ckpt_sf=u8(R * I // 16), codes=u8(R, 2 * I), sf=u8(R * I // 16),
            sf_layout=c, perm_src=i32(R), dgate_up=f32(R, 2 * I))),
        "moe_grouped_gemm_mxfp8": (moe.moe_grouped_gemm_mxfp8, dict(
            a_codes=u8(128, K), a_sf=u8(512), counts=i32(G), offsets=i32(G + 1), w_codes=u8(G, N, K // 2),
            w_sf=u8(G * 512), out=f32(128, N), status=i32(1))),
    }


# arguments whose type is the call's own: another one reaches the library, which refuses it
OWN_TYPE = {("moe_route_scores", "logits"), ("moe_swiglu_mxfp8", "gate_up"), ("moe_grouped_gemm_mxfp8", "out")}


@pytest.fixture
def stand(monkeypatch):
    return install(monkeypatch)


def refused(stand, f, args):
    del stand.calls[:]
    with pytest.raises(moe.MoEError):
        f(**args)
    assert not stand.calls


@pytest.mark.parametrize("name", sorted(calls()))
def test_fitting_arguments_reach_the_library(stand, name):
    f, args = calls()[name]
    f(**args)
    assert [c[0] for c in stand.calls] == [name]
    assert len(stand.calls[0][1]) == len(moe.SIGNATURES[name][1])


@pytest.mark.parametrize("name", sorted(calls()))
def test_other_types_sizes_and_strides_are_refused(stand, name):
    f, args = calls()[name]
    for arg, t in args.items():
        if not isinstance(t, torch.Tensor) or arg == "ws":
            continue
        for dt in (torch.float64, torch.int64, torch.int8):
            if (name, arg) in OWN_TYPE:
                assert moe._DTYPES[dt] < 0
                continue
            refused(stand, f, dict(args, **{arg: t.to(dt)}))
        wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)
        if t.numel() > 1:
            refused(stand, f, dict(args, **{arg: wide[..., ::2]}))
        if arg == "status":
            refused(stand, f, dict(args, status=i32(0)))
        elif ((name, arg) not in OWN_TYPE or arg == "out") and arg != "offsets":   # (more offsets fit)
            refused(stand, f, dict(args, **{arg: wide}))


@pytest.mark.parametrize("name", sorted(calls()))
def test_tensors_of_another_device_are_refused(stand, name, monkeypatch):
    f, args = calls()[name]
    monkeypatch.setattr(moe, "_place", lambda stream: (0, 0))
    refused(stand, f, args)
    monkeypatch.setattr(moe, "_place", lambda stream: (CPU, 0))

    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 0

    for arg, t in args.items():
        if isinstance(t, torch.Tensor):
            refused(stand, f, dict(args, **{arg: t.as_subclass(Elsewhere)}))


def test_outputs_that_belong_together(stand):
    f, args = calls()["moe_rmsnorm"]
    refused(stand, f, dict(args, sf=None))
    refused(stand, f, dict(args, codes=None))
    f, args = calls()["moe_swiglu_mxfp8"]
    refused(stand, f, dict(args, ckpt=None))
    f, args = calls()["moe_swiglu_mxfp8_backward"]
    refused(stand, f, dict(args, sf=None))
    f, args = calls()["moe_grouped_gemm_mxfp8"]
    refused(stand, f, dict(args, counts=None))


def test_sizes_past_32_bits_are_refused(stand):
    wide = torch.empty(1, dtype=torch.uint8).expand(2, 2 ** 31)
    for f, args in ((moe.moe_quant_mxfp8, dict(x=wide, codes=wide, sf=u8(1), sf_layout=0)),
                    (moe.moe_route_scores, dict(logits=torch.empty(1).expand(2 ** 31, 1), topk_ids=i32(1, 1).expand(2 ** 31, 1),
                                                topk_w=f32(1, 1)))):
        refused(stand, f, args)
