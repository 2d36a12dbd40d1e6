"""The gradient of softmax scores that are not renormalised where one score is nearly all: what is left of
the differences of the weights' gradients, relative to the result."""
import numpy as np
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
import ops8_ref as ref
from test_gpu_route_scores import DT, UNIT, W_TOL, dev

pytestmark = pytest.mark.gpu


def dense_grad(l, ids, dw, scale):
    """(gradient, the magnitudes that its terms add up to) of one token in 64 bits: with a_e the sum of an
    expert's gradients, p_e (sum_j p_j (a_e - a_j)) over all experts j."""
    E = len(l)
    s = ref.scores(l, "softmax")
    a = np.zeros(E)
    live = (ids >= 0) & (ids < E)
    np.add.at(a, ids[live].astype(np.int64), dw[live] * scale)
    d = a[:, None] - a[None, :]
    return s * (d * s).sum(1), s * (np.abs(d) * s).sum(1)


def check(l, ids, dw, dtype, scale=1.5):
    l = dev(l, DT[dtype])
    dw = np.float32(dw)
    out = torch.empty_like(l)
    moe.moe_route_scores_backward(l, dev(ids, torch.int32), dev(dw), out, score=moe.MOE_SCORE_SOFTMAX,
                                  renormalise=False, scale=scale)
    got, l64 = out.double().cpu().numpy(), l.double().cpu().numpy()
    for t in range(len(l64)):
        want, mag = dense_grad(l64[t], ids[t], dw[t].astype(np.float64), scale)
        # A score in front and scores in the sum, W_TOL each (of which roundings are a part).  Where the chosen
        # have up to 3/4 of the scores the sum may be a_e less sum_j p_j a_j: with |a_e| times the others' scores
        # at most mag and |a_j| at most |a_e| + |a_e - a_j|, that is of 3 mag + mag.  One rounding to the type.
        slack = 5 * W_TOL * mag + 2.0 ** -140
        step = 2.0 ** -25 if dtype == "fp16" else 0.0   # half of the smallest subnormal step
        assert np.all(np.abs(got[t] - want) <= slack + UNIT[dtype] * (np.abs(want) + slack) + step)
    return got


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,E,k", [(30, 320, 8), (30, 64, 1), (30, 1024, 32), (30, 9, 9), (30, 33, 2)])
def test_one_score_is_nearly_all(T, E, k, dtype):
    rng = np.random.default_rng(E)
    l = rng.normal(size=(T, E))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    # the raised expert is chosen, but for every fifth token (where another one, if there is any, is)
    for t in range(T):
        l[t, ids[t, t % k] if t % 5 else (ids[t, -1] + 1) % E] += (8, 12, 16, 18, 20, 24)[t % 6]
    got = check(l, ids, rng.normal(size=(T, k)), dtype)
    if dtype == "fp32":   # and so the row adds up to what rounding leaves of its terms
        assert np.all(np.abs(got.sum(1)) <= (5 * W_TOL + E * 2.0 ** -24) * np.abs(got).sum(1))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_the_same_expert_twice_and_ids_out_of_range(dtype):
    rng = np.random.default_rng(7)
    T, E = 12, 40
    l = rng.normal(size=(T, E))
    l[:, 3] += 17
    l[5:, 20:] = -np.inf
    ids = np.array([[3, 3, 8, 3], [8, 8, 3, -1], [40, 3, 2000000000, 3], [-1, -1, 41, 50]] * 3)
    check(l, ids, rng.normal(size=(T, 4)), dtype)
    check(l, ids, np.ones((T, 4)), dtype)


@pytest.mark.parametrize("renorm", [False, True])
def test_gradients_of_weights_next_to_each_other(renorm):
    """An expert of a small score whose weight's gradient is the nearly certain expert's up to 1e-5: their difference
    is exact before the scale, and rounded by it after."""
    T, E = 64, 24
    rng = np.random.default_rng(5)
    l = np.float32(rng.normal(size=(T, E)))
    l[:, 2] += 18
    ids = np.tile([2, 7, 11], (T, 1))
    dw = np.float32(rng.normal(size=(T, 3)))
    dw[:, 1] = dw[:, 0] * (1 + np.float32(2e-5) * np.float32(rng.uniform(-1, 1, size=T)))
    scale = 1.7
    out = torch.empty(T, E, device="cuda")
    moe.moe_route_scores_backward(dev(l), dev(ids, torch.int32), dev(dw), out, score=moe.MOE_SCORE_SOFTMAX,
                                  renormalise=renorm, scale=scale)
    got = out.double().cpu().numpy()
    for t in range(T):
        row = l[t].astype(np.float64)
        if renorm:
            row = np.where(np.isin(np.arange(E), ids[t]), row, -np.inf)   # the same as scores of the chosen alone
        want, mag = dense_grad(row, ids[t], dw[t].astype(np.float64), float(np.float32(scale)))
        assert np.all(np.abs(got[t] - want) <= 5 * W_TOL * mag + 2.0 ** -140)
