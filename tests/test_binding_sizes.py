"""Sizes past 32 bits: the C side takes int32, and a larger size, cut to 32 bits on the way, would be
another call (2^32 + 5 tokens: 5).  The tensors are without memory (meta), the library a stand-in."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
from stand_in import install

PAST = (2 ** 31, 2 ** 32 + 32)


@pytest.fixture
def lib(monkeypatch):
    s = install(monkeypatch)
    assert torch.empty(1, device="meta").get_device() == -1   # as the stand-in's current device
    return s


def m(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="meta")


def i32(*shape):
    return m(*shape, dtype=torch.int32)


def u8(*shape):
    return m(*shape, dtype=torch.uint8)


def dispatch(T=4, H=2, cap=8):
    moe.moe_dispatch(m(T, H), i32(T, 1), 4, 0, 4, 1, i32(4), i32(5), i32(cap), i32(T), m(cap, H))


def back(T=4, H=2, cap=8):
    moe.moe_dispatch_backward(m(cap, H), i32(T), 1, m(T, H))


def combine(T=4, H=2, cap=8):
    moe.moe_combine_weighted(m(cap, H), i32(T), m(T, 1), m(T, H))


def combine_back(T=4, H=2, cap=8):
    moe.moe_combine_backward(m(T, H), m(cap, H), i32(T), m(T, 1), m(cap, H), m(T, 1))


def quant(rows=4, cols=32):
    moe.moe_quant_mxfp4(m(rows, cols), u8(rows, cols // 2), u8(rows, cols // 32), moe.MOE_SF_CANONICAL)


def quant_t(rows=32, cols=4):
    moe.moe_quant_mxfp4(m(rows, cols), u8(cols, rows // 2), u8(cols, rows // 32), moe.MOE_SF_CANONICAL,
                        transpose=True)


def tile_scales(rows=4, cols=32, batch=1):
    tiled = batch * ((rows + 127) // 128) * ((cols + 127) // 128) * 512
    moe.moe_mxfp4_tile_scales(u8(batch, rows, cols // 32), batch, rows, cols, u8(tiled))


def product(cap=4, N=8, K=32, G=1):
    atoms = lambda rows: (rows + 127) // 128 * ((K + 127) // 128) * 512  # noqa: E731
    moe.moe_grouped_gemm_mxfp4(u8(cap, K // 2), u8(atoms(cap)), i32(G), i32(G), u8(G, N, K // 2),
                               u8(G * atoms(N)), m(cap, N))


CASES = [(dispatch, "T"), (dispatch, "H"), (dispatch, "cap"), (back, "T"), (back, "H"), (back, "cap"),
         (combine, "T"), (combine, "H"), (combine, "cap"), (combine_back, "T"), (combine_back, "H"),
         (combine_back, "cap"), (quant, "rows"), (quant, "cols"), (quant_t, "rows"), (quant_t, "cols"),
         (tile_scales, "rows"), (tile_scales, "cols"), (tile_scales, "batch"), (product, "cap"),
         (product, "N"), (product, "K"), (product, "G")]


@pytest.mark.parametrize("f,size", CASES, ids=["%s-%s" % (f.__name__, s) for f, s in CASES])
def test_sizes_past_32_bits_are_refused(lib, f, size):
    f()
    assert len(lib.calls) == 1
    for n in PAST:
        with pytest.raises(moe.MoEError):
            f(**{size: n})
    assert len(lib.calls) == 1


def test_sizing_of_sizes_past_32_bits_is_zero(lib):
    for n in PAST:
        assert moe.moe_dispatch_rows_capacity(n, 1, 4, 1) == 0
        for layout in (moe.MOE_SF_CANONICAL, moe.MOE_SF_TILED):
            assert moe.moe_mxfp4_scale_bytes(1, n, 32, layout) == 0
            assert moe.moe_mxfp4_scale_bytes(n, 1, 32, layout) == 0
            assert moe.moe_mxfp4_scale_bytes(1, 1, n, layout) == 0
