"""The norm's gradient where a warp or a block takes more than 32 rows (whose factors it holds 32 at a time),
several rows of 513 to 1024 16-bit elements a warp, and the weight's gradient past 2^31 elements, against 64 bits."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
import ops_ref

pytestmark = pytest.mark.gpu
EPS = 1e-6



def close(dy, h, dh, w, rstd, dx, dw, dtype, rows_of_a_part):
    """dx of the rows given, and dw of all, in 64 bits on the device; the bounds of the tests of fewer rows."""
    d, x64, r = dy.double(), h.double(), rstd.double()[:, None]
    wd = w.double()
    x = x64 * r
    mean = (d * wd * x).mean(1, keepdim=True)
    absd, absx = (d * wd).abs(), x.abs()
    want = r * (d * wd - x * mean) + dh.double()
    mag = (absd * absx).mean(1, keepdim=True)
    slack = r * (4 * 2.0 ** -24 * absd + 36 * 2.0 ** -24 * absx * mag)
    slack = slack + 2.0 ** -23 * (dh.double().abs() + r * (absd + absx * mag))
    unit = ops_ref.UNIT[dtype]
    assert torch.all((dx.double() - want).abs() <= unit * (want.abs() + slack) + slack + ops_ref.STEP[dtype])
    if dw is not None:
        # the rows of a part one after the other, eight warps, then at most 43 parts a thread, 32 threads
        n = rows_of_a_part + 8 + 43 + 5 + 2
        off = (dw.double() - (d * x).sum(0)).abs()
        assert torch.all(off <= n * 2.0 ** -24 * (d.abs() * absx).sum(0) + 1e-37)


# (fp32 of 520: a block a row, 1368 of them)
@pytest.mark.parametrize("T,H,dtype", [(80000, 64, "bf16"), (80000, 40, "fp32"), (80000, 512, "fp16"), (80000, 520, "bf16"),
                                       (5000, 1024, "fp16"), (50000, 520, "fp32"), (12000, 4096, "bf16"),
                                       (80000, 33, "bf16"), (12000, 4097, "fp16")])
def test_more_than_32_rows_a_warp_or_block(T, H, dtype):
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[dtype]
    g = torch.Generator("cuda").manual_seed(H)
    dy, h, dh = (torch.randn(T, H, generator=g, device="cuda").to(dt) for _ in range(3))
    w = torch.randn(H, generator=g, device="cuda").to(dt)
    # (factors that differ from row to row by more than rounding hides)
    h *= torch.linspace(0.5, 2, T, device="cuda").to(dt)[:, None]
    rstd = (1 / (h.double().square().mean(1) + EPS).sqrt()).float()
    ws = torch.empty(moe.moe_rmsnorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(dy), torch.empty(H, device="cuda")
    moe.moe_rmsnorm_backward(dy, h, w, rstd, dx, dw, ws, dh=dh)
    close(dy, h, dh, w, rstd, dx, dw, dtype, -(-T // 152))
    again, dx2 = torch.empty_like(dw), torch.empty_like(dx)
    moe.moe_rmsnorm_backward(dy, h, w, rstd, dx2, again, ws, dh=dh)
    assert torch.equal(dw, again) and torch.equal(dx, dx2)


def test_weight_gradient_past_2_31_elements():
    """Rows of zeros but for a few: their sum is the few rows' alone, in whatever parts they are."""
    T, H, at = 132000, 16384, [0, 1, 65537, 131071, 131072, 131999]
    g = torch.Generator("cuda").manual_seed(1)
    dy, h = (torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (dy, h):
        t[at] = torch.randn(len(at), H, generator=g, device="cuda").bfloat16()
    rstd = torch.rand(T, generator=g, device="cuda") + 0.5
    w = torch.randn(H, generator=g, device="cuda").bfloat16()
    ws = torch.empty(moe.moe_rmsnorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(dy), torch.empty(H, device="cuda")
    moe.moe_rmsnorm_backward(dy, h, w, rstd, dx, dw, ws)
    terms = dy[at].double() * h[at].double() * rstd[at].double()[:, None]
    # two roundings of a term, and at most five of the sum
    assert torch.all((dw.double() - terms.sum(0)).abs() <= 7 * 2.0 ** -24 * terms.abs().sum(0))
    close(dy[at], h[at], torch.zeros_like(dy[at]), w, rstd[at], dx[at], None, "bf16", 0)
    del ws, dy, h, dx
    torch.cuda.empty_cache()
