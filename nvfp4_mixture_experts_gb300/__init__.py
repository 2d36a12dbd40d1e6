"""Python binding of libnvfp4moe.so, the NVFP4 fused mixture-of-experts layer forward.

Argument marshalling only: every function forwards to the C entry point of the same name
(declared in include/nvfp4moe.h).  Tensors are torch tensors on the GPU (torch provides
device memory and streams); every step of the computation runs in the library's CUDA
kernels.  Importing raises if the compiled library is missing -- there is no fallback.
"""
import ctypes as C
import operator
import os

import torch

from . import build as _build

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = _build.LIB

MOE_OK, MOE_ERR_INVALID, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_WORKSPACE, \
    MOE_ERR_TIMEOUT, MOE_ERR_DEVICE_STATUS = range(7)
MOE_W4A4_DYNAMIC, MOE_W4A4_STATIC, MOE_W4A16 = 0, 1, 2
MOE_GS_ENCODE, MOE_GS_DEQUANT = 0, 1
MOE_TILING_AUTO, MOE_TILING_ROWS, MOE_TILING_TOKENS, MOE_TILING_PAIRS, MOE_TILING_WIDE = \
    0, 1, 2, 3, 4
MOE_DEV_BAD_EXPERT_ID, MOE_DEV_WAIT_TIMEOUT, MOE_DEV_ROWS_OVERFLOW = 1, 2, 4
MOE_DEV_BAD_INDEX = 8
MOE_BF16, MOE_FP16, MOE_FP32 = 0, 1, 2
MOE_SF_CANONICAL, MOE_SF_TILED = 0, 1
MOE_MX_FLOOR, MOE_MX_CEIL = 0, 1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP2 = 0, 1


class moe_config(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("inter", C.c_int32), ("num_experts", C.c_int32),
                ("top_k", C.c_int32), ("num_local_experts", C.c_int32),
                ("local_expert_offset", C.c_int32), ("has_shared", C.c_int32),
                ("shared_inter", C.c_int32), ("add_shared", C.c_int32),
                ("act_mode", C.c_int32), ("act_global_scale", C.c_float),
                ("inter_global_scale", C.c_float), ("max_tokens", C.c_int32),
                ("gemm_tiling", C.c_int32)]


class moe_weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "router_w_d", "w13_d", "w13_sf_d", "w13_gs_d", "w2_d", "w2_sf_d", "w2_gs_d",
        "sh13_d", "sh13_sf_d", "sh13_gs_d", "sh2_d", "sh2_sf_d", "sh2_gs_d")]


class _Int:
    """Argument type of a C int32: the interpreter's own conversion of an integer (ctypes', through an
    object of its own, takes five times as long: 19 arguments, 9 of them these, 2.1 -> 1.3 us)."""
    from_param = operator.index


_V = C.c_void_p
_I = _Int
_L = C.c_int64
_F = C.c_float
_SZ = C.c_size_t

# name -> (restype, argtypes); the list mirrors include/nvfp4moe.h
SIGNATURES = {
    "moe_create": (C.c_int, [C.POINTER(moe_config), C.POINTER(moe_weights), _V, C.POINTER(_V)]),
    "moe_destroy": (None, [_V]),
    "moe_workspace_size": (_SZ, [C.POINTER(moe_config), _I]),
    "moe_rows_capacity": (C.c_int32, [C.POINTER(moe_config), _I]),
    "moe_route_topk": (C.c_int, [_V, _V, _V, _V, _I, _V, _V, _V, _V, _SZ, _V]),
    "moe_route_topk_noalloc": (C.c_int, [_V, _V, _V, _V, _I, _V, _V, _V, _V]),
    "moe_permute": (C.c_int, [_V, _V, _I, _V, _V, _V, _V, _V, _SZ, _V]),
    "moe_quant_nvfp4": (C.c_int, [_V, _I, _I, _V, _V, _V, _V, _I, _V, _SZ, _V]),
    "moe_gather_activations": (C.c_int, [_V, _V, _I, _V, _V, _V, _V, _V, _V, _V, _SZ, _V]),
    "moe_grouped_gemm_gateup": (C.c_int, [_V, _V, _V, _V, _V, _V, _V, _I, _V, _V, _V, _V, _I,
                                          _V, _SZ, _V]),
    "moe_swiglu_requant": (C.c_int, [_V, _I, _I, C.c_float, _V, _V, _I, _V]),
    "moe_prepare_weights": (C.c_int, [_V, _V, _V, _I, _I, _I, _I, C.c_float, _I, _I, _I, _V,
                                      _V, _V, _V]),
    "moe_grouped_gemm_down": (C.c_int, [_V, _V, _V, _V, _V, _V, _V, _V, _V, _I, _V, _SZ, _V]),
    "moe_combine": (C.c_int, [_V, _V, _V, _V, _I, _V, _V]),
    "moe_forward": (C.c_int, [_V, _V, _V, _V, _I, _V, _V, _SZ, _V]),
    "moe_forward_host": (C.c_int, [_V, _V, _V, _V, _I, _V, _V, _SZ, _V]),
    "moe_workspace_size_host": (_SZ, [C.POINTER(moe_config), _I]),
    "moe_forward_buffers": (C.c_int, [_V, _V, _I] + [C.POINTER(_V)] * 16),
    "moe_get_status": (C.c_int, [_V, _V, _V, C.POINTER(C.c_uint32)]),
    "moe_status_string": (C.c_char_p, [C.c_int]),
    "moe_selftest_bounded_wait": (C.c_int, [_V, C.c_uint64, _V]),
    "moe_selftest_group_wait": (C.c_int, [_V, C.c_uint64, _V]),
    "moe_dispatch_rows_capacity": (C.c_int32, [_I] * 4),
    "moe_dispatch": (C.c_int, [_V, _I, _L, _V] + [_I] * 8 + [_V] * 7),
    "moe_dispatch_backward": (C.c_int, [_V, _I, _V] + [_I] * 4 + [_V, _L, _V]),
    "moe_combine_weighted": (C.c_int, [_V, _I, _V, _V] + [_I] * 4 + [_V, _L, _V]),
    "moe_combine_backward": (C.c_int, [_V, _I, _L, _V, _V, _V] + [_I] * 4 + [_V, _V, _V]),
    "moe_mxfp4_scale_bytes": (_SZ, [_I] * 4),
    "moe_quant_mxfp4": (C.c_int, [_V] + [_I] * 4 + [_L, _L, _I, _I, _V, _V, _V, _I, _V, _V]),
    "moe_mxfp4_tile_scales": (C.c_int, [_V, _I, _I, _I, _V, _V]),
    "moe_mxfp4_workspace_size": (_SZ, [_I] * 4),
    "moe_grouped_gemm_mxfp4": (C.c_int, [_V, _V, _I, _V, _V, _I, _V, _V, _I, _I, _V, _I, _L, _V,
                                         _SZ, _V, _V]),
    "moe_route_scores": (C.c_int, [_V, _I, _L, _V] + [_I] * 8 + [_F, _V, _V, _V]),
    "moe_route_scores_backward": (C.c_int, [_V, _I, _L, _V, _V] + [_I] * 5 + [_F, _V, _L, _V]),
    "moe_rmsnorm": (C.c_int, [_V, _I, _L, _V, _L, _V, _F, _I, _I, _V, _L, _V, _L, _V, _V, _V, _I, _I,
                              _V]),
    "moe_rmsnorm_workspace_size": (_SZ, [_I] * 2),
    "moe_rmsnorm_backward": (C.c_int, [_V, _I, _L, _V, _L, _V, _L, _V, _V, _I, _I, _V, _L, _V, _V, _SZ,
                                       _V]),
    "moe_quant_mxfp8": (C.c_int, [_V] + [_I] * 4 + [_L, _L, _I, _V, _V, _V, _I, _V, _V]),
    "moe_swiglu_mxfp8": (C.c_int, [_V, _I, _L, _I, _I, _V, _I, _V, _V, _I, _V, _V, _V]),
    "moe_swiglu_mxfp8_backward": (C.c_int, [_V, _I, _L, _V, _V, _I, _I, _V, _I, _V, _V, _I, _V, _V]),
    "moe_grouped_gemm_mxfp8": (C.c_int, [_V, _V, _I, _V, _V, _I, _V, _V, _I, _I, _V, _I, _L, _V, _V]),
}

_lib = None
_lib_debug = None


def _open(p):
    if not os.path.exists(p):
        raise OSError("%s not built: run __graft_entry__.build()" % p)
    lib = C.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


def load(path=None):
    """Loads the compiled library (raises OSError if it is not there)."""
    global _lib
    if _lib is None:
        _lib = _open(path or LIB_PATH)
    return _lib


def load_debug():
    """The MOE_DEBUG flavour of the library (same entry points; every index read from a
    buffer is bounds-checked on the device and a bad one flags MOE_DEV_BAD_INDEX).  Handles
    of one flavour are used with that flavour's calls only."""
    global _lib_debug
    if _lib_debug is None:
        _lib_debug = _open(_build.LIB_DEBUG)
    return _lib_debug


class MoEError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = load().moe_status_string(status).decode()
        super().__init__("%s: %s (%d)" % (where, msg, status))


def _check(status, where):
    if status != MOE_OK:
        raise MoEError(status, where)


def _p(t):
    """Device pointer of a torch tensor (or None)."""
    return None if t is None else t.data_ptr()


_cuda = None  # torch._C, bound at the first call


def _stream(stream):
    """The handle of a torch stream, of an integer, or (None) of the current stream."""
    if stream is None:
        global _cuda
        if _cuda is None:
            torch.cuda.current_stream()  # the CUDA context exists
            _cuda = torch._C
        return _cuda._cuda_getCurrentRawStream(_cuda._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _place(stream):
    """(device, stream handle) of a launch: the current device, on which the tensors and a stream
    given as a torch stream have to be (device -2, which no tensor has, for a stream that is not)."""
    if stream is None and _cuda is not None:
        dev = _cuda._cuda_getDevice()
        return dev, _cuda._cuda_getCurrentRawStream(dev)
    handle = _stream(stream)
    dev = torch._C._cuda_getDevice()
    return (dev if stream is None or getattr(stream, "device_index", dev) == dev else -2), handle


# ---------------------------------------------------------------- C entry points

def moe_create(cfg, weights, stream=None):
    h = C.c_void_p()
    _check(load().moe_create(C.byref(cfg), C.byref(weights), _stream(stream), C.byref(h)),
           "moe_create")
    return h


def moe_destroy(h):
    load().moe_destroy(h)


def moe_workspace_size(cfg, T):
    return load().moe_workspace_size(C.byref(cfg), T)


def moe_rows_capacity(cfg, T):
    return load().moe_rows_capacity(C.byref(cfg), T)


def moe_route_topk(h, x, logits_in, logit_bias, T, topk_ids, topk_w, logits_out, ws,
                   stream=None):
    _check(load().moe_route_topk(h, _p(x), _p(logits_in), _p(logit_bias), T, _p(topk_ids),
                                 _p(topk_w), _p(logits_out), _p(ws),
                                 0 if ws is None else ws.numel() * ws.element_size(),
                                 _stream(stream)), "moe_route_topk")


def moe_route_topk_noalloc(h, x, logits_in, logit_bias, T, topk_ids, topk_w, logits_out,
                           stream=None):
    """moe_route_topk without a workspace: the scratch is a static device array of the
    library (see include/nvfp4moe.h for its size limit and sharing rules)."""
    _check(load().moe_route_topk_noalloc(h, _p(x), _p(logits_in), _p(logit_bias), T,
                                         _p(topk_ids), _p(topk_w), _p(logits_out),
                                         _stream(stream)), "moe_route_topk_noalloc")


def moe_permute(h, topk_ids, T, counts, offsets, perm_src, inv, ws, stream=None):
    _check(load().moe_permute(h, _p(topk_ids), T, _p(counts), _p(offsets), _p(perm_src),
                              _p(inv), _p(ws), ws.numel() * ws.element_size(),
                              _stream(stream)), "moe_permute")


def moe_quant_nvfp4(x, rows, cols, gs_in, gs_out, codes, sf, sf_layout, ws, stream=None):
    _check(load().moe_quant_nvfp4(_p(x), rows, cols, _p(gs_in), _p(gs_out), _p(codes), _p(sf),
                                  sf_layout, _p(ws),
                                  0 if ws is None else ws.numel() * ws.element_size(),
                                  _stream(stream)), "moe_quant_nvfp4")


def moe_gather_activations(h, x, T, inv, offsets, a_codes, a_sf, a_bf16, gs_out, ws,
                           stream=None):
    _check(load().moe_gather_activations(h, _p(x), T, _p(inv), _p(offsets), _p(a_codes),
                                         _p(a_sf), _p(a_bf16), _p(gs_out), _p(ws),
                                         ws.numel() * ws.element_size(), _stream(stream)),
           "moe_gather_activations")


def moe_grouped_gemm_gateup(h, a_codes, a_sf, gs_a, a_bf16, counts, offsets, fuse_epilogue,
                            gateup_f32, inter_codes, inter_sf, inter_bf16, T, ws, stream=None):
    _check(load().moe_grouped_gemm_gateup(h, _p(a_codes), _p(a_sf), _p(gs_a), _p(a_bf16),
                                          _p(counts), _p(offsets), int(fuse_epilogue),
                                          _p(gateup_f32), _p(inter_codes), _p(inter_sf),
                                          _p(inter_bf16), T, _p(ws),
                                          ws.numel() * ws.element_size(), _stream(stream)),
           "moe_grouped_gemm_gateup")


def moe_swiglu_requant(gateup_f32, rows, inter, gs_i, codes, sf, sf_layout, stream=None):
    _check(load().moe_swiglu_requant(_p(gateup_f32), rows, inter, float(gs_i), _p(codes),
                                     _p(sf), sf_layout, _stream(stream)), "moe_swiglu_requant")


def moe_prepare_weights(codes, sf, glob, N, K, convention, fold_target, swap_halves, off, count,
                        codes_out, sf_out, gs_out, stream=None):
    _check(load().moe_prepare_weights(_p(codes), _p(sf), _p(glob), int(glob.numel()), N, K,
                                      convention, float(fold_target), int(bool(swap_halves)),
                                      off, count, _p(codes_out), _p(sf_out), _p(gs_out),
                                      _stream(stream)), "moe_prepare_weights")


def moe_grouped_gemm_down(h, inter_codes, inter_sf, inter_bf16, counts, offsets, perm_src,
                          topk_w, y, T, ws, stream=None):
    _check(load().moe_grouped_gemm_down(h, _p(inter_codes), _p(inter_sf), _p(inter_bf16),
                                        _p(counts), _p(offsets), _p(perm_src), _p(topk_w),
                                        _p(y), T, _p(ws), ws.numel() * ws.element_size(),
                                        _stream(stream)), "moe_grouped_gemm_down")


def moe_combine(h, y, inv, offsets, T, out, stream=None):
    _check(load().moe_combine(h, _p(y), _p(inv), _p(offsets), T, _p(out), _stream(stream)),
           "moe_combine")


def moe_forward(h, x, logits_in, logit_bias, T, out, ws, stream=None):
    _check(load().moe_forward(h, _p(x), _p(logits_in), _p(logit_bias), T, _p(out), _p(ws),
                              ws.numel() * ws.element_size(), _stream(stream)), "moe_forward")


def moe_forward_host(h, x_host, logits_in, logit_bias, T, out_host, ws, stream=None):
    """x_host / out_host: CPU tensors (pinned for asynchronous copies); ws: a device workspace
    of moe_workspace_size_host bytes."""
    _check(load().moe_forward_host(h, _p(x_host), _p(logits_in), _p(logit_bias), T,
                                   _p(out_host), _p(ws), ws.numel() * ws.element_size(),
                                   _stream(stream)), "moe_forward_host")


def moe_workspace_size_host(cfg, T):
    return load().moe_workspace_size_host(C.byref(cfg), T)


FORWARD_BUFFERS = ("topk_ids", "topk_w", "expert_counts", "expert_offsets", "perm_src", "inv",
                   "gs_a", "a_codes", "a_sf", "a_bf16", "inter_codes", "inter_sf", "inter_bf16",
                   "y", "inter_gs", "y_scale")


def moe_forward_buffers(h, ws, T):
    """Device addresses (ints) of moe_forward's intermediates inside ws."""
    ptrs = [C.c_void_p() for _ in FORWARD_BUFFERS]
    _check(load().moe_forward_buffers(h, _p(ws), T, *[C.byref(p) for p in ptrs]),
           "moe_forward_buffers")
    return {n: p.value for n, p in zip(FORWARD_BUFFERS, ptrs)}


def moe_selftest_bounded_wait(status_word, limit_ns, stream=None):
    """Runs the bounded-wait failure self-test (status_word: a device tensor of >= 4 bytes);
    returns the status code (MOE_ERR_TIMEOUT expected)."""
    return load().moe_selftest_bounded_wait(_p(status_word), int(limit_ns), _stream(stream))


def moe_selftest_group_wait(words, limit_ns, stream=None):
    """Runs the self-test of a wait that runs out in one warp of a group (words: a device tensor
    of >= 8 bytes); returns the status code (MOE_ERR_TIMEOUT expected)."""
    return load().moe_selftest_group_wait(_p(words), int(limit_ns), _stream(stream))


def moe_get_status(h, ws, stream=None):
    bits = C.c_uint32(0)
    st = load().moe_get_status(h, _p(ws), _stream(stream), C.byref(bits))
    return st, bits.value


# ---------------------------------------------------------------- operators without a handle
# Element types come from the tensors (int16 tensors are bf16 bit patterns, as above), sizes from
# their shapes; a tensor whose type, shape, strides or device do not fit raises MoEError before the
# call: the C side sees addresses alone.  Ids, maps, counts and status words are int32, codes and
# scales uint8, all contiguous; every tensor is on the current device.  (Small calls are bound by this
# side: each tensor's attributes are asked for once.)

class _Dtypes(dict):
    """torch dtype -> moe_dtype (-1: none)."""

    def __missing__(self, key):
        return -1


_DTYPES = _Dtypes({torch.bfloat16: MOE_BF16, torch.int16: MOE_BF16, torch.float16: MOE_FP16,
                   torch.float32: MOE_FP32})
_I32, _U8, _F32 = torch.int32, torch.uint8, torch.float32
# Integers are 32-bit numbers on the C side, to which a larger one would be cut: an or of them is negative or
# passes this if one is or does.
_MOST = 0x7fffffff


def _refuse(where):
    raise MoEError(MOE_ERR_INVALID, where)


def _sf_bytes(batch, rows, blocks, sf_layout):
    """moe_mxfp4_scale_bytes for `blocks` scales a row (-1, no tensor's, for another layout)."""
    if sf_layout == MOE_SF_TILED:
        return batch * ((rows + 127) >> 7) * ((blocks + 3) >> 2) * 512
    return batch * rows * blocks if sf_layout == MOE_SF_CANONICAL else -1


def moe_dispatch_rows_capacity(T, k, num_local, row_align):
    if not 0 <= (T | k | num_local | row_align) <= _MOST:
        return 0
    return load().moe_dispatch_rows_capacity(T, k, num_local, row_align)


def moe_dispatch(x, topk_ids, num_experts, local_off, num_local, row_align, counts, offsets,
                 perm_src, inv, rows, status=None, stream=None):
    """x [T, H] (None: the maps alone, rows None too), topk_ids int32 [T, k]; outputs counts
    [num_local], offsets [num_local + 1], perm_src [rows_cap], inv [T * k] (all int32), rows
    [rows_cap, H]; status: an int32 word that errors found on the device are or-ed into."""
    T, k = topk_ids.shape
    cap = perm_src.numel()
    if not (0 <= (T | k | cap | num_experts | local_off | num_local | row_align) <= _MOST and
            topk_ids.dtype is _I32 and topk_ids.is_contiguous() and
            inv.dtype is _I32 and inv.numel() == T * k and inv.is_contiguous() and
            counts.dtype is _I32 and counts.numel() == num_local and counts.is_contiguous() and
            offsets.dtype is _I32 and offsets.numel() == num_local + 1 and
            offsets.is_contiguous() and perm_src.dtype is _I32 and perm_src.is_contiguous() and
            (status is None or (status.dtype is _I32 and status.numel())) and
            (x is None) == (rows is None)):
        _refuse("moe_dispatch")
    H, xs, dt, px, pr = 1, 1, MOE_BF16, None, None
    if x is not None:
        Tx, H = x.shape
        xs, one = x.stride()
        dt = _DTYPES[x.dtype]
        rows_cap, Hr = rows.shape
        if not (Tx == T and H <= _MOST and (one == 1 or H == 1 or T == 0) and dt == _DTYPES[rows.dtype] and
                rows_cap == cap and Hr == H and rows.is_contiguous()):
            _refuse("moe_dispatch")
        px, pr = x.data_ptr(), rows.data_ptr()
    dev, handle = _place(stream)
    if not (dev == topk_ids.get_device() == inv.get_device() == counts.get_device() ==
            offsets.get_device() == perm_src.get_device() and
            (x is None or dev == x.get_device() == rows.get_device()) and
            (status is None or status.get_device() == dev)):
        _refuse("moe_dispatch")
    st = (_lib or load()).moe_dispatch(
        px, dt, xs, topk_ids.data_ptr(), T, k, H, num_experts, local_off, num_local, row_align,
        cap, counts.data_ptr(), offsets.data_ptr(), perm_src.data_ptr(), inv.data_ptr(), pr,
        _p(status), handle)
    if st:
        _check(st, "moe_dispatch")


def moe_dispatch_backward(drows, inv, k, dx, stream=None):
    """drows [rows_cap, H], inv int32 [T * k] -> dx [T, H]."""
    T, H = dx.shape
    cap, Hr = drows.shape
    xs, one = dx.stride()
    dt = _DTYPES[dx.dtype]
    if not (Hr == H and 0 <= (T | H | cap | k) <= _MOST and (one == 1 or H == 1 or T == 0) and
            drows.is_contiguous() and _DTYPES[drows.dtype] == dt and inv.dtype is _I32 and inv.numel() == T * k and
            inv.is_contiguous()):
        _refuse("moe_dispatch_backward")
    dev, handle = _place(stream)
    if not dev == drows.get_device() == inv.get_device() == dx.get_device():
        _refuse("moe_dispatch_backward")
    st = (_lib or load()).moe_dispatch_backward(drows.data_ptr(), dt, inv.data_ptr(), T, k, H, cap,
                                                dx.data_ptr(), xs, handle)
    if st:
        _check(st, "moe_dispatch_backward")


def moe_combine_weighted(y, inv, w, out, stream=None):
    """y [rows_cap, H], inv int32 [T * k], w float32 [T, k] -> out [T, H]."""
    T, k = w.shape
    To, H = out.shape
    cap, Hy = y.shape
    xs, one = out.stride()
    dt = _DTYPES[y.dtype]
    if not (To == T and Hy == H and (T | k | H | cap) <= _MOST and (one == 1 or H == 1 or T == 0) and
            y.is_contiguous() and
            _DTYPES[out.dtype] == dt and inv.dtype is _I32 and inv.numel() == T * k and
            inv.is_contiguous() and w.is_contiguous() and w.dtype is _F32):
        _refuse("moe_combine_weighted")
    dev, handle = _place(stream)
    if not dev == y.get_device() == inv.get_device() == w.get_device() == out.get_device():
        _refuse("moe_combine_weighted")
    st = (_lib or load()).moe_combine_weighted(y.data_ptr(), dt, inv.data_ptr(), w.data_ptr(), T, k,
                                               H, cap, out.data_ptr(), xs, handle)
    if st:
        _check(st, "moe_combine_weighted")


def moe_combine_backward(dout, y, inv, w, dy, dw, stream=None):
    """dout [T, H], y [rows_cap, H], inv int32 [T * k], w float32 [T, k] -> dy [rows_cap, H] and
    dw float32 [T, k]; dy or dw may be None (and y with dw)."""
    T, k = w.shape
    To, H = dout.shape
    xs, one = dout.stride()
    dt = _DTYPES[dout.dtype]
    ok = (To == T and (one == 1 or H == 1 or T == 0) and inv.dtype is _I32 and inv.numel() == T * k and
          inv.is_contiguous() and w.is_contiguous() and w.dtype is _F32)
    ok = ok and not (dy is None and dw is None) and (T | k | H) <= _MOST
    cap = None
    for t in (y, dy):
        if t is not None:
            rows, Ht = t.shape
            ok = (ok and Ht == H and rows <= _MOST and t.is_contiguous() and _DTYPES[t.dtype] == dt and
                  (cap is None or cap == rows))
            cap = rows
    if dw is not None:
        ok = (ok and dw.numel() == T * k and dw.is_contiguous() and
              dw.dtype is _F32 and y is not None)
    if not ok:
        _refuse("moe_combine_backward")
    dev, handle = _place(stream)
    if not (dev == dout.get_device() == inv.get_device() == w.get_device() and
            (y is None or y.get_device() == dev) and (dy is None or dy.get_device() == dev) and
            (dw is None or dw.get_device() == dev)):
        _refuse("moe_combine_backward")
    st = (_lib or load()).moe_combine_backward(dout.data_ptr(), dt, xs, _p(y), inv.data_ptr(),
                                               w.data_ptr(), T, k, H, cap or 0, _p(dy), _p(dw),
                                               handle)
    if st:
        _check(st, "moe_combine_backward")


def moe_mxfp4_scale_bytes(batch, rows, cols, sf_layout):
    if not 0 <= (batch | rows | cols | sf_layout) <= _MOST:
        return 0
    return load().moe_mxfp4_scale_bytes(batch, rows, cols, sf_layout)


def _quant(where, per, x, codes, sf, sf_layout, transpose, scale_rule, perm_src, values, stream):
    """The arguments that moe_quant_mxfp4 (per: two codes a byte) and moe_quant_mxfp8 (one) begin with,
    checked: x's, and the stream's handle."""
    shape, stride = x.shape, x.stride()
    if len(shape) == 3:
        (B, R, Cc), (bs, rs, one) = shape, stride
    elif len(shape) == 2:
        (R, Cc), (rs, one) = shape, stride
        B, bs = 1, 0
    else:
        _refuse(where)
    n, dt = B * R * Cc, _DTYPES[x.dtype]
    scales = _sf_bytes(B, Cc, R >> 5, sf_layout) if transpose else _sf_bytes(B, R, Cc >> 5, sf_layout)
    if not (0 <= (B | R | Cc | scale_rule) <= _MOST and (one == 1 or Cc == 1 or n == 0) and codes.dtype is _U8 and
            codes.numel() * per == n and codes.is_contiguous() and sf.dtype is _U8 and
            sf.numel() == scales and sf.is_contiguous() and
            (perm_src is None or (perm_src.dtype is _I32 and perm_src.numel() == R and
                                  perm_src.is_contiguous())) and
            (values is None or (values.numel() == n and values.is_contiguous() and
                                _DTYPES[values.dtype] == dt))):
        _refuse(where)
    dev, handle = _place(stream)
    if not (dev == x.get_device() == codes.get_device() == sf.get_device() and
            (perm_src is None or perm_src.get_device() == dev) and
            (values is None or values.get_device() == dev)):
        _refuse(where)
    return (x.data_ptr(), dt, B, R, Cc, rs, bs), handle


def moe_quant_mxfp4(x, codes, sf, sf_layout, transpose=False, scale_rule=MOE_MX_FLOOR,
                    perm_src=None, values=None, stream=None):
    """x [rows, cols] or [batch, rows, cols] (columns contiguous); codes uint8, sf uint8 and values
    (x's type) hold the MXFP4 matrix, or with transpose that of each matrix's transpose."""
    args, handle = _quant("moe_quant_mxfp4", 2, x, codes, sf, sf_layout, transpose, scale_rule, perm_src,
                          values, stream)
    st = (_lib or load()).moe_quant_mxfp4(*args, 1 if transpose else 0, scale_rule, _p(perm_src),
                                          codes.data_ptr(), sf.data_ptr(), sf_layout, _p(values), handle)
    if st:
        _check(st, "moe_quant_mxfp4")


def moe_quant_mxfp8(x, codes, sf, sf_layout, scale_rule=MOE_MX_CEIL, perm_src=None, values=None,
                    stream=None):
    """x [rows, cols] or [batch, rows, cols] (columns contiguous) -> codes uint8 of x's shape and sf
    uint8, its MXFP8 matrix, and values (x's type; None)."""
    args, handle = _quant("moe_quant_mxfp8", 1, x, codes, sf, sf_layout, False, scale_rule, perm_src, values,
                          stream)
    st = (_lib or load()).moe_quant_mxfp8(*args, scale_rule, _p(perm_src), codes.data_ptr(),
                                          sf.data_ptr(), sf_layout, _p(values), handle)
    if st:
        _check(st, "moe_quant_mxfp8")


def moe_mxfp4_tile_scales(sf, batch, rows, cols, sf_tiled, stream=None):
    if not (0 <= (batch | rows | cols) <= _MOST and
            sf.numel() == _sf_bytes(batch, rows, cols >> 5, MOE_SF_CANONICAL) and
            sf_tiled.numel() == _sf_bytes(batch, rows, cols >> 5, MOE_SF_TILED) and
            sf.is_contiguous() and sf_tiled.is_contiguous() and sf.dtype is _U8 and
            sf_tiled.dtype is _U8):
        _refuse("moe_mxfp4_tile_scales")
    dev, handle = _place(stream)
    if not dev == sf.get_device() == sf_tiled.get_device():
        _refuse("moe_mxfp4_tile_scales")
    st = (_lib or load()).moe_mxfp4_tile_scales(_p(sf), batch, rows, cols, _p(sf_tiled), handle)
    if st:
        _check(st, "moe_mxfp4_tile_scales")


def moe_mxfp4_workspace_size(rows_cap, num_groups, N, K):
    if not 0 <= (rows_cap | num_groups | N | K) <= _MOST:
        return 0
    return load().moe_mxfp4_workspace_size(rows_cap, num_groups, N, K)


def _product(where, per, a_codes, a_sf, counts, offsets, w_codes, w_sf, out, ws, status, stream):
    """The arguments that moe_grouped_gemm_mxfp4 (per: two codes of a byte in the rows) and
    moe_grouped_gemm_mxfp8 (one) begin with, checked, and the stream's handle."""
    G, N, K2 = w_codes.shape
    cap, Ka = a_codes.shape
    rows, No = out.shape
    xs, one = out.stride()
    if not (Ka * per == 2 * K2 and (cap | G | N | 2 * K2) <= _MOST and a_codes.is_contiguous() and
            w_codes.is_contiguous() and a_codes.dtype is _U8 and w_codes.dtype is _U8 and
            a_sf.dtype is _U8 and a_sf.numel() == _sf_bytes(1, cap, K2 >> 4, MOE_SF_TILED) and
            a_sf.is_contiguous() and
            w_sf.dtype is _U8 and w_sf.numel() == _sf_bytes(G, N, K2 >> 4, MOE_SF_TILED) and
            w_sf.is_contiguous() and
            rows == cap and No == N and (one == 1 or N == 1 or cap == 0) and
            (counts is None) == (offsets is None) and
            (counts is None or (counts.dtype is _I32 and counts.numel() == G and
                                counts.is_contiguous() and offsets.dtype is _I32 and
                                offsets.numel() >= G and offsets.is_contiguous())) and
            (ws is None or ws.is_contiguous()) and
            (status is None or (status.dtype is _I32 and status.numel()))):
        _refuse(where)
    dev, handle = _place(stream)
    if not (dev == a_codes.get_device() == a_sf.get_device() == w_codes.get_device() ==
            w_sf.get_device() == out.get_device() and
            (counts is None or dev == counts.get_device() == offsets.get_device()) and
            (ws is None or ws.get_device() == dev) and
            (status is None or status.get_device() == dev)):
        _refuse(where)
    return (a_codes.data_ptr(), a_sf.data_ptr(), cap, _p(counts), _p(offsets), G, w_codes.data_ptr(),
            w_sf.data_ptr(), N, 2 * K2, out.data_ptr(), _DTYPES[out.dtype], xs), handle


def moe_grouped_gemm_mxfp4(a_codes, a_sf, counts, offsets, w_codes, w_sf, out, ws=None,
                           status=None, stream=None):
    """a_codes [rows_cap, K/2], w_codes [num_groups, N, K/2] (uint8) with tiled scales; counts and
    offsets int32 (both None: one group, all rows); out [rows_cap, N]."""
    args, handle = _product("moe_grouped_gemm_mxfp4", 2, a_codes, a_sf, counts, offsets, w_codes, w_sf,
                            out, ws, status, stream)
    st = (_lib or load()).moe_grouped_gemm_mxfp4(*args, _p(ws), 0 if ws is None else ws.nbytes,
                                                 _p(status), handle)
    if st:
        _check(st, "moe_grouped_gemm_mxfp4")


def moe_grouped_gemm_mxfp8(a_codes, a_sf, counts, offsets, w_codes, w_sf, out, status=None, stream=None):
    """a_codes [rows_cap, K], w_codes [num_groups, N, K/2] (uint8) with tiled scales; counts and
    offsets int32 (both None: one group, all rows); out [rows_cap, N]."""
    args, handle = _product("moe_grouped_gemm_mxfp8", 1, a_codes, a_sf, counts, offsets, w_codes, w_sf,
                            out, None, status, stream)
    st = (_lib or load()).moe_grouped_gemm_mxfp8(*args, _p(status), handle)
    if st:
        _check(st, "moe_grouped_gemm_mxfp8")


def _row_stride(t, shape, dt, dev):
    """The row stride of a tensor of rows of this shape, moe_dtype and device with contiguous columns, or -1."""
    if t.shape != shape or _DTYPES[t.dtype] != dt or t.get_device() != dev:
        return -1
    stride, one = t.stride()
    return stride if one == 1 or shape[1] == 1 or shape[0] == 0 else -1


def _flat(t, n, dtype):
    """Whether t is n contiguous elements of a torch dtype."""
    return t.dtype is dtype and t.numel() == n and t.is_contiguous()


def moe_route_scores(logits, topk_ids, topk_w, bias=None, score=MOE_SCORE_SOFTMAX, num_groups=1,
                     topk_groups=1, group_score=MOE_GROUP_MAX, renormalise=True, scale=1.0, stream=None):
    """logits [T, num_experts], bias float32 [num_experts] (None) -> topk_ids int32 [T, k], topk_w
    float32 [T, k]."""
    T, E = logits.shape
    Tk, k = topk_ids.shape
    stride, one = logits.stride()
    if not (Tk == T and 0 <= (T | E | k | score | num_groups | topk_groups | group_score) <= _MOST and
            (one == 1 or E == 1 or T == 0) and
            topk_ids.dtype is _I32 and topk_ids.is_contiguous() and _flat(topk_w, T * k, _F32) and
            (bias is None or _flat(bias, E, _F32))):
        _refuse("moe_route_scores")
    dev, handle = _place(stream)
    if not (dev == logits.get_device() == topk_ids.get_device() == topk_w.get_device() and
            (bias is None or bias.get_device() == dev)):
        _refuse("moe_route_scores")
    st = (_lib or load()).moe_route_scores(
        logits.data_ptr(), _DTYPES[logits.dtype], stride, _p(bias), T, E, k, score, num_groups, topk_groups,
        group_score, 1 if renormalise else 0, scale, topk_ids.data_ptr(), topk_w.data_ptr(), handle)
    if st:
        _check(st, "moe_route_scores")


def moe_route_scores_backward(logits, topk_ids, dtopk_w, dlogits, score=MOE_SCORE_SOFTMAX,
                              renormalise=True, scale=1.0, stream=None):
    """logits [T, num_experts], topk_ids int32 [T, k], dtopk_w float32 [T, k] -> dlogits (logits' type)
    [T, num_experts]."""
    shape = logits.shape
    T, E = shape
    Tk, k = topk_ids.shape
    stride, one = logits.stride()
    dt = _DTYPES[logits.dtype]
    if not (Tk == T and 0 <= (T | E | k | score) <= _MOST and (one == 1 or E == 1 or T == 0) and
            topk_ids.dtype is _I32 and topk_ids.is_contiguous() and _flat(dtopk_w, T * k, _F32)):
        _refuse("moe_route_scores_backward")
    dev, handle = _place(stream)
    ds = _row_stride(dlogits, shape, dt, dev)
    if not (ds >= 0 and dev == logits.get_device() == topk_ids.get_device() == dtopk_w.get_device()):
        _refuse("moe_route_scores_backward")
    st = (_lib or load()).moe_route_scores_backward(
        logits.data_ptr(), dt, stride, topk_ids.data_ptr(), dtopk_w.data_ptr(), T, E, k, score,
        1 if renormalise else 0, scale, dlogits.data_ptr(), ds, handle)
    if st:
        _check(st, "moe_route_scores_backward")


def moe_rmsnorm(x, weight, eps, residual=None, h=None, y=None, rstd=None, codes=None, sf=None,
                sf_layout=MOE_SF_TILED, scale_rule=MOE_MX_CEIL, stream=None):
    """x [T, H], weight [H] (None: ones), residual [T, H] (None) -> any of h, y [T, H] (x's type), rstd
    float32 [T], and codes [T, H] with sf (uint8), y's MXFP8 matrix."""
    shape, xt = x.shape, x.dtype
    T, H = shape
    xs, one = x.stride()
    dt = _DTYPES[xt]
    dev, handle = _place(stream)
    ok = (0 <= (T | H | sf_layout | scale_rule) <= _MOST and (one == 1 or H == 1 or T == 0) and
          x.get_device() == dev)
    pr = ph = py = pw = ps = pc = pf = None
    rs = hs = ys = 0
    if weight is not None:
        ok = ok and _flat(weight, H, xt) and weight.get_device() == dev
        pw = weight.data_ptr()
    if residual is not None:
        pr, rs = residual.data_ptr(), _row_stride(residual, shape, dt, dev)
    if h is not None:
        ph, hs = h.data_ptr(), _row_stride(h, shape, dt, dev)
    if y is not None:
        py, ys = y.data_ptr(), _row_stride(y, shape, dt, dev)
    ok = ok and rs >= 0 and hs >= 0 and ys >= 0
    if rstd is not None:
        ok = ok and _flat(rstd, T, _F32) and rstd.get_device() == dev
        ps = rstd.data_ptr()
    if codes is not None or sf is not None:
        ok = (ok and codes is not None and sf is not None and _flat(codes, T * H, _U8) and
              _flat(sf, _sf_bytes(1, T, H >> 5, sf_layout), _U8) and
              dev == codes.get_device() == sf.get_device())
        pc, pf = _p(codes), _p(sf)
    if not ok:
        _refuse("moe_rmsnorm")
    st = (_lib or load()).moe_rmsnorm(x.data_ptr(), dt, xs, pr, rs, pw, eps, T, H, ph, hs, py, ys, ps, pc, pf,
                                      sf_layout, scale_rule, handle)
    if st:
        _check(st, "moe_rmsnorm")


def moe_rmsnorm_workspace_size(T, H):
    if not 0 <= (T | H) <= _MOST:
        return 0
    return load().moe_rmsnorm_workspace_size(T, H)


def moe_rmsnorm_backward(dy, h, weight, rstd, dx, dweight=None, ws=None, dh=None, stream=None):
    """dy, h [T, H], weight [H] (None: ones), rstd float32 [T], dh [T, H] (None) -> dx [T, H] and
    dweight float32 [H] (None); ws: moe_rmsnorm_workspace_size bytes where dweight is given."""
    shape = dy.shape
    T, H = shape
    stride, one = dy.stride()
    dt = _DTYPES[dy.dtype]
    dev, handle = _place(stream)
    es = 0 if dh is None else _row_stride(dh, shape, dt, dev)
    hs, xs = _row_stride(h, shape, dt, dev), _row_stride(dx, shape, dt, dev)
    if not ((T | H) <= _MOST and (one == 1 or H == 1 or T == 0) and es >= 0 and hs >= 0 and xs >= 0 and
            dev == dy.get_device() == rstd.get_device() and _flat(rstd, T, _F32) and
            (weight is None or (_flat(weight, H, dy.dtype) and weight.get_device() == dev)) and
            (dweight is None or (_flat(dweight, H, _F32) and dweight.get_device() == dev)) and
            (ws is None or (ws.is_contiguous() and ws.get_device() == dev))):
        _refuse("moe_rmsnorm_backward")
    st = (_lib or load()).moe_rmsnorm_backward(
        dy.data_ptr(), dt, stride, _p(dh), es, h.data_ptr(), hs,
        _p(weight), rstd.data_ptr(), T, H, dx.data_ptr(), xs, _p(dweight), _p(ws),
        0 if ws is None else ws.nbytes, handle)
    if st:
        _check(st, "moe_rmsnorm_backward")


def moe_swiglu_mxfp8(gate_up, codes, sf, sf_layout, ckpt=None, ckpt_sf=None, perm_src=None,
                     scale_rule=MOE_MX_CEIL, stream=None):
    """gate_up [rows, 2 * inter] -> codes [rows, inter] with sf (uint8), silu(gate) * up as an MXFP8
    matrix, and ckpt [rows, 2 * inter] with canonical scales ckpt_sf (None), that of gate_up."""
    R, I2 = gate_up.shape
    stride, one = gate_up.stride()
    I = I2 >> 1
    if not (0 <= (R | I2 | sf_layout | scale_rule) <= _MOST and not I2 & 1 and (one == 1 or R == 0) and
            _flat(codes, R * I, _U8) and
            _flat(sf, _sf_bytes(1, R, I >> 5, sf_layout), _U8) and (ckpt is None) == (ckpt_sf is None) and
            (ckpt is None or (_flat(ckpt, R * I2, _U8) and _flat(ckpt_sf, R * (I2 >> 5), _U8))) and
            (perm_src is None or _flat(perm_src, R, _I32))):
        _refuse("moe_swiglu_mxfp8")
    dev, handle = _place(stream)
    if not (dev == gate_up.get_device() == codes.get_device() == sf.get_device() and
            (ckpt is None or dev == ckpt.get_device() == ckpt_sf.get_device()) and
            (perm_src is None or perm_src.get_device() == dev)):
        _refuse("moe_swiglu_mxfp8")
    st = (_lib or load()).moe_swiglu_mxfp8(
        gate_up.data_ptr(), _DTYPES[gate_up.dtype], stride, R, I, _p(perm_src), scale_rule, codes.data_ptr(),
        sf.data_ptr(), sf_layout, _p(ckpt), _p(ckpt_sf), handle)
    if st:
        _check(st, "moe_swiglu_mxfp8")


def moe_swiglu_mxfp8_backward(ds, ckpt, ckpt_sf, codes=None, sf=None, sf_layout=MOE_SF_TILED,
                              perm_src=None, dgate_up=None, scale_rule=MOE_MX_CEIL, stream=None):
    """ds [rows, inter] and the checkpoint of moe_swiglu_mxfp8 -> codes [rows, 2 * inter] with sf
    (uint8), gate_up's gradient as an MXFP8 matrix, and/or dgate_up [rows, 2 * inter] in ds's type."""
    R, I = ds.shape
    stride, one = ds.stride()
    dt = _DTYPES[ds.dtype]
    if not (0 <= (R | 2 * I | sf_layout | scale_rule) <= _MOST and (one == 1 or I == 1 or R == 0) and
            _flat(ckpt, 2 * R * I, _U8) and
            _flat(ckpt_sf, R * (2 * I >> 5), _U8) and (codes is None) == (sf is None) and
            (codes is None or (_flat(codes, 2 * R * I, _U8) and
                               _flat(sf, _sf_bytes(1, R, 2 * I >> 5, sf_layout), _U8))) and
            (dgate_up is None or (_DTYPES[dgate_up.dtype] == dt and dgate_up.numel() == 2 * R * I and
                                  dgate_up.is_contiguous())) and
            (perm_src is None or _flat(perm_src, R, _I32))):
        _refuse("moe_swiglu_mxfp8_backward")
    dev, handle = _place(stream)
    if not (dev == ds.get_device() == ckpt.get_device() == ckpt_sf.get_device() and
            (codes is None or dev == codes.get_device() == sf.get_device()) and
            (dgate_up is None or dgate_up.get_device() == dev) and
            (perm_src is None or perm_src.get_device() == dev)):
        _refuse("moe_swiglu_mxfp8_backward")
    st = (_lib or load()).moe_swiglu_mxfp8_backward(
        ds.data_ptr(), dt, stride, ckpt.data_ptr(), ckpt_sf.data_ptr(), R, I, _p(perm_src), scale_rule,
        _p(codes), _p(sf), sf_layout, _p(dgate_up), handle)
    if st:
        _check(st, "moe_swiglu_mxfp8_backward")


from .layer import MoELayer, make_config  # noqa: E402,F401
