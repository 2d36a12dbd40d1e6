"""Argument checks of the handle-free operators: answered on the host, before any launch (the
pointers given here are never read)."""
import ctypes as C

import pytest

import nvfp4_mixture_experts_gb300 as moe
from nvfp4_mixture_experts_gb300 import build as moe_build

P = C.c_void_p(4096)      # a well aligned address that nothing reads
ODD = C.c_void_p(4104)
BYTE = C.c_void_p(4097)   # no multiple of an element's size


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


def call(lib, name, defaults, **kw):
    args = dict(defaults)
    assert set(kw) <= set(args), kw
    args.update(kw)
    return getattr(lib, name)(*args.values())


DISPATCH = dict(x=P, dtype=0, x_stride=64, ids=P, T=4, k=2, H=64, E=8, off=0, El=8, align=1,
                cap=8, counts=P, offsets=P, perm=P, inv=P, rows=P, status=None, stream=None)
COMBINE = dict(y=P, dtype=0, inv=P, w=P, T=4, k=2, H=64, cap=8, out=P, out_stride=64, stream=None)
BACK = dict(dout=P, dtype=0, stride=64, y=P, inv=P, w=P, T=4, k=2, H=64, cap=8, dy=P, dw=P,
            stream=None)
QUANT = dict(x=P, dtype=0, batch=1, rows=4, cols=64, rs=64, bs=0, transpose=0, rule=0, perm=None,
             codes=P, sf=P, layout=1, values=None, stream=None)
GEMM = dict(a=P, a_sf=P, cap=128, counts=P, offsets=P, G=2, w=P, w_sf=P, N=64, K=64, out=P,
            dtype=0, stride=64, ws=None, ws_bytes=0, status=None, stream=None)

INVALID = [
    ("moe_dispatch", DISPATCH, [dict(dtype=3), dict(T=-1), dict(k=0), dict(H=0), dict(cap=-1),
                                dict(E=0), dict(off=-1), dict(El=9), dict(off=1), dict(align=3),
                                dict(align=256), dict(align=0), dict(k=9), dict(x_stride=63),
                                dict(x=None), dict(rows=None), dict(ids=None), dict(counts=None),
                                dict(offsets=None), dict(perm=None), dict(inv=None),
                                dict(x=BYTE), dict(rows=BYTE)]),
    ("moe_dispatch_backward", {k: v for k, v in COMBINE.items() if k != "w"},
     [dict(dtype=-1), dict(T=-1), dict(k=0), dict(H=0), dict(inv=None), dict(out=None),
      dict(y=None), dict(out_stride=63)]),
    ("moe_combine_weighted", COMBINE, [dict(dtype=3), dict(w=None), dict(y=None), dict(inv=None),
                                       dict(out=None), dict(out_stride=1), dict(cap=-1),
                                       dict(y=BYTE), dict(out=BYTE), dict(out=C.c_void_p(4098), dtype=2)]),
    ("moe_combine_backward", BACK, [dict(dtype=3), dict(dout=None), dict(inv=None), dict(w=None),
                                    dict(dy=None, dw=None), dict(y=None), dict(stride=63),
                                    dict(dout=BYTE), dict(y=BYTE), dict(dy=BYTE)]),
    ("moe_quant_mxfp4", QUANT, [dict(dtype=3), dict(batch=-1), dict(rows=-1), dict(cols=0),
                                dict(transpose=2), dict(rule=2), dict(layout=2), dict(x=None),
                                dict(codes=None), dict(sf=None), dict(rs=63), dict(codes=ODD),
                                dict(values=ODD), dict(x=BYTE), dict(sf=ODD), dict(perm=P, batch=2),
                                dict(perm=P, transpose=1, rows=32)]),
    ("moe_grouped_gemm_mxfp4", GEMM,
     [dict(dtype=3), dict(cap=-1), dict(G=0), dict(N=0), dict(K=0), dict(counts=None),
      dict(offsets=None), dict(counts=None, offsets=None), dict(a=None), dict(a_sf=None),
      dict(w=None), dict(w_sf=None), dict(out=None), dict(stride=63), dict(a=ODD), dict(a_sf=ODD),
      dict(w=ODD), dict(w_sf=ODD), dict(ws=ODD), dict(ws_bytes=1), dict(out=C.c_void_p(4097))]),
]
UNSUPPORTED = [
    ("moe_dispatch", DISPATCH, [dict(k=33, E=64), dict(E=2000), dict(T=2 ** 30, k=4)]),
    ("moe_combine_weighted", COMBINE, [dict(k=33), dict(T=2 ** 30, k=4)]),
    ("moe_combine_backward", BACK, [dict(k=33)]),
    ("moe_quant_mxfp4", QUANT, [dict(cols=48, rs=48), dict(transpose=1, rows=33)]),
    ("moe_grouped_gemm_mxfp4", GEMM, [dict(K=48), dict(G=1025), dict(G=1024, N=2 ** 22)]),
]
NOTHING = [  # nothing to do: no pointer is needed
    ("moe_dispatch_backward", {k: v for k, v in COMBINE.items() if k != "w"}, dict(T=0, y=None, inv=None, out=None)),
    ("moe_combine_weighted", COMBINE, dict(T=0, y=None, inv=None, w=None, out=None)),
    ("moe_combine_backward", BACK, dict(T=0, dout=None, y=None, inv=None, w=None)),
    ("moe_quant_mxfp4", QUANT, dict(rows=0, x=None, codes=None, sf=None)),
    ("moe_grouped_gemm_mxfp4", GEMM, dict(cap=0, a=None, a_sf=None, out=None)),
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


def test_sizes(lib):
    cap = moe.moe_dispatch_rows_capacity
    assert cap(1, 8, 320, 128) == 8 * 128 and cap(5, 3, 4, 1) == 15 and cap(0, 2, 4, 8) == 0
    assert cap(100, 2, 3, 16) == (200 + 3 * 15 + 15) // 16 * 16
    assert cap(-1, 2, 4, 1) == 0 and cap(4, 33, 4, 1) == 0 and cap(4, 2, 4, 3) == 0
    assert cap(2 ** 30, 4, 4, 1) == 0
    sb = moe.moe_mxfp4_scale_bytes
    assert sb(2, 5, 64, moe.MOE_SF_CANONICAL) == 20
    assert sb(2, 129, 160, moe.MOE_SF_TILED) == 2 * 2 * 2 * 512
    assert sb(1, 1, 48, 0) == 0 and sb(1, 1, 64, 2) == 0
    assert moe.moe_mxfp4_workspace_size(128, 4, 256, 64) <= 32 << 20
    assert moe.moe_mxfp4_workspace_size(128, 0, 256, 64) == 0


def test_binding_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    x, i32 = torch.zeros(4, 64), dict(dtype=torch.int32)
    ids, inv, w = torch.zeros(4, 2, **i32), torch.zeros(8, **i32), torch.zeros(4, 2)
    y, out = torch.zeros(8, 64), torch.zeros(4, 64)
    bad = [
        lambda: moe.moe_dispatch(x, ids, 8, 0, 8, 1, torch.zeros(7, **i32), torch.zeros(9, **i32),
                                 torch.zeros(8, **i32), inv, y),
        lambda: moe.moe_dispatch(x, ids, 8, 0, 8, 1, torch.zeros(8, **i32), torch.zeros(9, **i32),
                                 torch.zeros(8, **i32), inv, y.half()),
        lambda: moe.moe_dispatch(x.t().contiguous().t(), ids, 8, 0, 8, 1, torch.zeros(8, **i32),
                                 torch.zeros(9, **i32), torch.zeros(8, **i32), inv, y),
        lambda: moe.moe_combine_weighted(y.half(), inv, w, out),
        lambda: moe.moe_combine_weighted(y, inv, w.half(), out),
        lambda: moe.moe_combine_weighted(y, inv[:7], w, out),
        lambda: moe.moe_dispatch_backward(y, inv, 2, out.double()),
        lambda: moe.moe_combine_backward(out, y[:7], inv, w, y, w),
        lambda: moe.moe_quant_mxfp4(x, torch.zeros(4, 31, dtype=torch.uint8),
                                    torch.zeros(512, dtype=torch.uint8), moe.MOE_SF_TILED),
        lambda: moe.moe_grouped_gemm_mxfp4(torch.zeros(128, 32, dtype=torch.uint8),
                                           torch.zeros(512, dtype=torch.uint8), None, None,
                                           torch.zeros(1, 64, 16, dtype=torch.uint8),
                                           torch.zeros(512, dtype=torch.uint8),
                                           torch.zeros(128, 64)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(moe.MoEError):
            f()
