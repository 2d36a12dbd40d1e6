"""Bounded waits of warps that work together."""
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe


@pytest.mark.gpu
def test_a_group_of_warps_gives_up_together():
    """One warp's wait runs out where its group's other waits end well: all four leave, the other
    group goes on, and the context stays usable."""
    words = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    for _ in range(3):
        assert moe.moe_selftest_group_wait(words, 2 * 10 ** 6) == moe.MOE_ERR_TIMEOUT
        assert words.tolist() == [moe.MOE_DEV_WAIT_TIMEOUT, 0xF0]


def test_limits_out_of_range_are_refused():
    from nvfp4_mixture_experts_gb300 import build as moe_build
    moe_build.build()
    lib = moe.load()
    for words, limit in ((None, 1000), (4096, 0), (4096, 3 * 10 ** 9), (4098, 1000)):
        assert lib.moe_selftest_group_wait(words, limit, None) == moe.MOE_ERR_INVALID
