"""The first CUDA work of a host thread may be a call of this library."""
import threading

import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu


def in_a_new_thread(f):
    result = []

    def run():
        try:
            result.append(f())
        except Exception as e:
            result.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    if isinstance(result[0], Exception):
        raise result[0]
    return result[0]


def test_product():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    a, sa, w, sw = u8(5, 16).fill_(0x22), u8(512).fill_(127), u8(1, 32, 16).fill_(0x44), u8(512).fill_(127)
    out, stream = torch.zeros(5, 32, device="cuda"), torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    in_a_new_thread(lambda: moe.moe_grouped_gemm_mxfp4(a, sa, None, None, w, sw, out, stream=stream))
    assert torch.all(out == 64.0)     # 32 products 1 x 2


@pytest.mark.parametrize("T", [8, 800])
def test_dispatch(T):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, counts, offs, perm, inv = i32(T, 2), i32(4), i32(5), i32(2 * T), i32(2 * T)
    x, rows, stream = torch.randn(T, 40, device="cuda"), torch.zeros(2 * T, 40, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    in_a_new_thread(lambda: moe.moe_dispatch(x, ids, 4, 0, 4, 1, counts, offs, perm, inv, rows, stream=stream))
    torch.cuda.synchronize()
    assert counts.tolist() == [2 * T, 0, 0, 0] and torch.equal(rows, x.repeat_interleave(2, 0))


@pytest.mark.parametrize("transpose", [False, True])
def test_quantiser(transpose):
    x = torch.ones(32, 32, device="cuda")
    codes = torch.zeros(32, 16, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(32, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    in_a_new_thread(lambda: moe.moe_quant_mxfp4(x, codes, sf, moe.MOE_SF_CANONICAL, transpose=transpose,
                                                stream=stream))
    torch.cuda.synchronize()
    assert torch.all(codes == 0x66) and torch.all(sf == 125)     # 1 = 4 x 2^-2
