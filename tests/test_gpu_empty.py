"""Sorted rows of no tokens, and of no capacity: a tensor without elements has no address."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu


def i32(*shape):
    return torch.full(shape, -7, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dispatch_of_no_tokens_into_rows_of_a_capacity(dtype):
    counts, offs, perm, inv = i32(3), i32(4), i32(40), i32(0)
    rows, status = torch.full((40, 24), -3.0, dtype=dtype, device="cuda"), torch.zeros_like(i32(1))
    x = torch.empty(0, 24, dtype=dtype, device="cuda")
    moe.moe_dispatch(x, i32(0, 2), 3, 0, 3, 8, counts, offs, perm, inv, rows, status)
    assert counts.tolist() == [0] * 3 and offs.tolist() == [0] * 4 and perm.tolist() == [-1] * 40
    assert torch.all(rows == -3.0) and status.item() == 0
    # and back: gradients and outputs of no tokens
    w = torch.empty(0, 2, device="cuda")
    dx, dw, dy = torch.empty_like(x), torch.empty_like(w), torch.full_like(rows, -3.0)
    moe.moe_dispatch_backward(rows, inv, 2, dx)
    moe.moe_combine_weighted(rows, inv, w, dx)
    moe.moe_combine_backward(x, rows, inv, w, dy, dw)
    assert torch.all(dy == -3.0)


@pytest.mark.parametrize("T", [5, 2000])
def test_rows_of_no_capacity(T):
    """Every pair is dropped and flagged; what comes back is zero."""
    counts, offs, perm, inv = i32(3), i32(4), i32(0), i32(2 * T)
    ids = torch.zeros_like(i32(T, 2))
    x, rows, status = torch.randn(T, 24, device="cuda"), torch.empty(0, 24, device="cuda"), torch.zeros_like(i32(1))
    moe.moe_dispatch(x, ids, 3, 0, 3, 1, counts, offs, perm, inv, rows, status)
    assert counts.tolist() == [2 * T, 0, 0] and torch.all(inv == -1)
    assert status.item() == moe.MOE_DEV_ROWS_OVERFLOW
    w, out, dw = torch.rand(T, 2, device="cuda"), torch.full_like(x, -3.0), torch.full((T, 2), -3.0, device="cuda")
    moe.moe_combine_weighted(rows, inv, w, out)
    assert torch.all(out == 0.0)
    out.fill_(-3.0)
    moe.moe_dispatch_backward(rows, inv, 2, out)
    assert torch.all(out == 0.0)
    moe.moe_combine_backward(x, rows, inv, w, torch.empty_like(rows), dw)
    assert torch.all(dw == 0.0)
    moe.moe_combine_backward(x, None, inv, w, torch.empty_like(rows), None)
