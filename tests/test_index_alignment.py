"""Arrays of 32-bit words (ids, maps, counts, weights, status) at addresses that are no multiple of
4 are refused on the host, as rows at no multiple of their element's size are: a kernel's access to
one is an error that takes the context with it."""
import ctypes as C

import pytest

import nvfp4_mixture_experts_gb300 as moe
from test_ops_refusals import BACK, COMBINE, DISPATCH, GEMM, P, QUANT, call, lib  # noqa: F401

ODD = [C.c_void_p(4096 + i) for i in (1, 2, 3)]
CASES = [
    ("moe_dispatch", DISPATCH, ("ids", "counts", "offsets", "perm", "inv", "status")),
    ("moe_dispatch_backward", {k: v for k, v in COMBINE.items() if k != "w"}, ("inv",)),
    ("moe_combine_weighted", COMBINE, ("inv", "w")),
    ("moe_combine_backward", BACK, ("inv", "w", "dw")),
    ("moe_quant_mxfp4", QUANT, ("perm",)),
    ("moe_grouped_gemm_mxfp4", GEMM, ("counts", "offsets", "status")),
]


@pytest.mark.parametrize("name,defaults,args", CASES, ids=[c[0] for c in CASES])
def test_word_arrays_are_words(lib, name, defaults, args):  # noqa: F811
    assert P.value % 16 == 0
    for arg in args:
        assert arg in defaults
        for odd in ODD:
            assert call(lib, name, defaults, **{arg: odd}) == moe.MOE_ERR_INVALID, (arg, odd)
