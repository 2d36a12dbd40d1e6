"""A launch that fails is reported by its own call alone."""
import ctypes as C

import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu


def test_a_failed_launch_leaves_no_error_behind():
    """A launch on the legacy stream is refused while a stream that synchronises with it is being
    captured (an error of the host's, nothing runs); the next call is then as any other."""
    rt = C.CDLL("libcudart.so.13")       # torch's; streams are the driver's
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, inv = torch.ones(4, 8, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda")
    dx = torch.zeros(4, 8, device="cuda")
    torch.cuda.synchronize()
    stream, graph, relaxed = C.c_void_p(), C.c_void_p(), 2
    assert rt.cudaStreamCreate(C.byref(stream)) == 0
    try:
        assert rt.cudaStreamBeginCapture(stream, relaxed) == 0
        with pytest.raises(moe.MoEError) as e:
            moe.moe_dispatch_backward(y, inv, 1, dx, stream=0)
        assert e.value.status == moe.MOE_ERR_CUDA
    finally:
        rt.cudaStreamEndCapture(stream, C.byref(graph))
        rt.cudaStreamDestroy(stream)
        rt.cudaGetLastError()
    assert moe.moe_selftest_bounded_wait(word, 10 ** 6) == moe.MOE_ERR_TIMEOUT
    moe.moe_dispatch_backward(y, inv, 1, dx)
    assert torch.equal(dx, y)
