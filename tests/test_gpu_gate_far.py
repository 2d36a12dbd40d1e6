"""The gate's gradient in fp32 for far gates: within what its sigmoid's comment states."""
import numpy as np
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
import ops8_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most", [5.0, 20.0, 80.0])
def test_gradient_of_far_gates(most):
    R, I = 64, 256
    rng = np.random.default_rng(int(most))
    gu = torch.from_numpy(np.concatenate([rng.uniform(-most, most, size=(R, I)), rng.normal(size=(R, I))], 1)).float().cuda()
    ck = torch.empty(R, 2 * I, dtype=torch.uint8, device="cuda")
    ck_sf = torch.empty(R, I // 16, dtype=torch.uint8, device="cuda")
    moe.moe_quant_mxfp8(gu, ck, ck_sf, moe.MOE_SF_CANONICAL)
    held = ref.decode8(ck.cpu().numpy(), ck_sf.cpu().numpy())
    g, u = held[:, :I], held[:, I:]
    assert np.abs(g).max() <= most * 1.0625
    ds = rng.normal(size=(R, I)).astype(np.float32).astype(np.float64)
    out = torch.empty(R, 2 * I, device="cuda")
    moe.moe_swiglu_mxfp8_backward(torch.from_numpy(ds).float().cuda(), ck, ck_sf, dgate_up=out)
    got = out.double().cpu().numpy()
    dg, du = ref.swiglu_grad(ds, g, u)
    s = ref.sigmoid(g)
    off = 2.0 ** -21 + 1.25 * np.abs(g) * 2.0 ** -24     # of the sigmoid, relative to it
    h = 2.0 ** -24
    # t = ds s and t g: two roundings; 1 - s is off by s off and a rounding, times g, and a rounding of the sum
    tiny = 2.0 ** -120    # (sigmoids below 2^-126 are 0)
    assert np.all(np.abs(got[:, I:] - du) <= np.abs(du) * (off + 3 * h) + tiny)
    inner = np.abs(g) * (s * off + h) + 2 * h * (1 + np.abs(g) * (1 - s))
    assert np.all(np.abs(got[:, :I] - dg) <= np.abs(dg) * (off + 5 * h) + np.abs(ds * u) * s * (1 + off) * inner + tiny)
