"""The binding of the handle-free operators hands nothing but addresses to the C side, so a tensor
of another type, layout or device than the call's has to stop in the binding.  A stand-in takes the
place of the library (no kernel runs): calls that fit reach it, the others raise before it."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
from nvfp4_mixture_experts_gb300 import build as moe_build

CPU = -1  # what a CPU tensor's get_device() gives


class StandIn:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return moe.MOE_OK
        return call

    @staticmethod
    def moe_status_string(status):
        return b"refused"


@pytest.fixture
def lib(monkeypatch):
    """The stand-in, with the CPU as the current device."""
    moe_build.build()
    moe.load()
    s = StandIn()
    monkeypatch.setattr(moe, "_lib", s)
    monkeypatch.setattr(moe, "_place", lambda stream: (CPU, 0), raising=False)
    monkeypatch.setattr(moe, "_stream", lambda stream: 0)
    return s


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def calls():
    """name -> (function, arguments that fit)."""
    T, H, k, E, cap = 4, 64, 2, 8, 16
    x, rows, w = torch.zeros(T, H), torch.zeros(cap, H), torch.zeros(T, k)
    G, N, K = 3, 32, 64
    return {
        "moe_dispatch": (moe.moe_dispatch, dict(
            x=x, topk_ids=i32(T, k), num_experts=E, local_off=0, num_local=E, row_align=1,
            counts=i32(E), offsets=i32(E + 1), perm_src=i32(cap), inv=i32(T * k), rows=rows,
            status=i32(1))),
        "moe_dispatch_backward": (moe.moe_dispatch_backward, dict(drows=rows, inv=i32(T * k), k=k, dx=x)),
        "moe_combine_weighted": (moe.moe_combine_weighted, dict(y=rows, inv=i32(T * k), w=w, out=x)),
        "moe_combine_backward": (moe.moe_combine_backward, dict(
            dout=x, y=rows, inv=i32(T * k), w=w, dy=torch.zeros(cap, H), dw=torch.zeros(T, k))),
        "moe_quant_mxfp4": (moe.moe_quant_mxfp4, dict(
            x=x, codes=u8(T, H // 2), sf=u8(T * H // 32), sf_layout=moe.MOE_SF_CANONICAL,
            perm_src=i32(T), values=torch.zeros(T, H))),
        "moe_mxfp4_tile_scales": (moe.moe_mxfp4_tile_scales, dict(
            sf=u8(T * H // 32), batch=1, rows=T, cols=H, sf_tiled=u8(512))),
        "moe_grouped_gemm_mxfp4": (moe.moe_grouped_gemm_mxfp4, dict(
            a_codes=u8(128, K // 2), a_sf=u8(512), counts=i32(G), offsets=i32(G + 1),
            w_codes=u8(G, N, K // 2), w_sf=u8(G * 512), out=torch.zeros(128, N), ws=u8(0),
            status=i32(1))),
    }


INTS = {"topk_ids", "counts", "offsets", "perm_src", "inv", "status"}
BYTES = {"codes", "sf", "sf_tiled", "a_codes", "a_sf", "w_codes", "w_sf"}


def strided(t):
    """The same shape and type, every element of the last axis two apart."""
    wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)
    return wide[..., ::2]


def refused(lib, f, args):
    del lib.calls[:]
    with pytest.raises(moe.MoEError):
        f(**args)
    assert not lib.calls


@pytest.mark.parametrize("name", sorted(calls()))
def test_fitting_arguments_reach_the_library(lib, name):
    f, args = calls()[name]
    f(**args)
    assert lib.calls == [name]


@pytest.mark.parametrize("name", sorted(calls()))
def test_other_types_are_refused(lib, name):
    f, args = calls()[name]
    for arg, t in args.items():
        if arg in INTS:
            others = (torch.int64, torch.int16, torch.uint8, torch.float32)
        elif arg in BYTES:
            others = (torch.int32, torch.int8, torch.float32)
        elif isinstance(t, torch.Tensor) and arg != "ws":
            others = (torch.float64, torch.int32, torch.uint8)
        else:
            continue
        if name == "moe_grouped_gemm_mxfp4" and arg == "out":
            continue  # its type is a value of the call, refused by the library
        if name == "moe_quant_mxfp4" and arg == "x":
            args = dict(args, values=None)
        for dt in others:
            bad = dict(args, **{arg: t.to(dt)})
            if arg == "x" and name == "moe_quant_mxfp4":
                assert moe._DTYPES[dt] < 0  # refused by the library
                continue
            refused(lib, f, bad)


@pytest.mark.parametrize("name", sorted(calls()))
def test_strided_arguments_are_refused(lib, name):
    f, args = calls()[name]
    for arg, t in args.items():
        if isinstance(t, torch.Tensor) and t.numel() > 1:
            refused(lib, f, dict(args, **{arg: strided(t)}))


@pytest.mark.parametrize("name", sorted(calls()))
def test_tensors_of_another_device_are_refused(lib, name, monkeypatch):
    """The CPU's tensors, all of them or one, where the call goes to device 0; and the reverse."""
    f, args = calls()[name]
    monkeypatch.setattr(moe, "_place", lambda stream: (0, 0), raising=False)
    refused(lib, f, args)
    monkeypatch.setattr(moe, "_place", lambda stream: (CPU, 0), raising=False)

    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 0

    for arg, t in args.items():
        if isinstance(t, torch.Tensor):
            refused(lib, f, dict(args, **{arg: t.as_subclass(Elsewhere)}))


def test_a_stream_of_another_device_is_refused(lib, monkeypatch):
    monkeypatch.undo()
    monkeypatch.setattr(moe, "_lib", lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)

    class Stream:
        cuda_stream = 7

        def __init__(self, device):
            self.device_index = device

    assert moe._place(Stream(0)) == (0, 7) and moe._place(7) == (0, 7)
    assert moe._place(Stream(1))[0] not in (0, 1, CPU)


def test_a_status_of_no_words_is_refused(lib):
    for name in ("moe_dispatch", "moe_grouped_gemm_mxfp4"):
        f, args = calls()[name]
        refused(lib, f, dict(args, status=i32(0)))
