"""The large sort in a cluster of the portable size, which the debug flavour always takes (the other
flavour where the device has none of twice the blocks): the same maps and rows."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
from nvfp4_mixture_experts_gb300 import build as moe_build

pytestmark = pytest.mark.gpu


def run(ids, x, E, off, El, align):
    T, k = ids.shape
    i32 = lambda n: torch.full((n,), -7, dtype=torch.int32, device="cuda")  # noqa: E731
    cap = moe.moe_dispatch_rows_capacity(T, k, El, align)
    out = [i32(El), i32(El + 1), i32(cap), i32(T * k), torch.full((cap, x.shape[1]), -3.0, device="cuda")]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_dispatch(x, ids, E, off, El, align, *out, status)
    return out + [status]


@pytest.mark.parametrize("T,E,k,off,El,align", [(513, 8, 2, 0, 8, 1), (3001, 320, 8, 160, 160, 128),
                                                (70001, 1024, 2, 0, 1024, 1), (131073, 7, 1, 2, 4, 4)])
def test_both_cluster_sizes_agree(T, E, k, off, El, align, monkeypatch):
    moe_build.build(debug=True)
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.randint(-1, E + 1, (T, k), generator=g, device="cuda", dtype=torch.int32)  # some out of range
    x = torch.randn(T, 12, generator=g, device="cuda")
    want = run(ids, x, E, off, El, align)
    monkeypatch.setattr(moe, "_lib", moe.load_debug())
    got = run(ids, x, E, off, El, align)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # the counts by definition
    le = ids.view(-1).long() - off
    assert torch.equal(got[0].long(), torch.bincount(le[(le >= 0) & (le < El) & (ids.view(-1) < E)], minlength=El))
    assert got[-1].item() == moe.MOE_DEV_BAD_EXPERT_ID
