"""Routing from logits (scores, bias, groups, top-k, weights) and the gradient of the logits, against
64-bit implementations of the definition."""
import numpy as np
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
import ops8_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
KIND = {"softmax": moe.MOE_SCORE_SOFTMAX, "sigmoid": moe.MOE_SCORE_SIGMOID}
# A weight: exponentials (2^-23 and their argument's rounding, |l| 2^-24 with |l| <= 32 here), a sum of at
# most 32 + 5 terms in a row (37 2^-24; of all logits of a lane as well), a division and a product
W_TOL = (2 * (2 + 32 + 37) + 4) * 2.0 ** -24


def dev(a, dt=torch.float32):
    return torch.as_tensor(a).to(dt).cuda()


def run(l, bias, k, kind, groups=1, topg=1, top2=False, renorm=True, scale=1.0, **kw):
    T = l.shape[0]
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    moe.moe_route_scores(l, ids, w, bias=bias, score=KIND[kind], num_groups=groups, topk_groups=topg,
                         group_score=moe.MOE_GROUP_TOP2 if top2 else moe.MOE_GROUP_MAX,
                         renormalise=renorm, scale=scale, **kw)
    return ids, w


def check(l, bias, k, kind, groups=1, topg=1, top2=False, renorm=True, scale=1.0):
    ids, w = run(l, bias, k, kind, groups, topg, top2, renorm, scale)
    b = None if bias is None else bias.double().cpu().numpy()
    want, ww = ref.route(l.double().cpu().numpy(), b, k, kind, groups, topg, top2, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), want)
    got = w.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ww))
    ok = ~np.isnan(ww)
    # (an unnormalised score may be a subnormal number of 32 bits)
    assert np.all(np.abs(got - ww)[ok] <= W_TOL * np.abs(ww)[ok] + 2.0 ** -140)


CASES = [  # T, E, k, groups, topg
    (1, 1, 1, 1, 1), (1, 320, 8, 1, 1), (5, 33, 32, 1, 1), (37, 64, 6, 8, 3), (130, 320, 8, 8, 4),
    (9, 256, 8, 1, 1), (64, 384, 4, 4, 4), (33, 1024, 32, 32, 7), (17, 60, 5, 3, 2), (3, 40, 1, 20, 1),
    (250, 100, 7, 5, 2), (6, 513, 9, 27, 26), (4, 32, 32, 32, 32), (2, 32, 32, 1, 1),
]


@pytest.mark.parametrize("T,E,k,groups,topg", CASES)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_choice_and_weights(T, E, k, groups, topg, kind, dtype):
    g = torch.Generator().manual_seed(E * 7 + k)
    l = dev(torch.randn(T, E + 3, generator=g) * 2, DT[dtype])[:, :E]   # strided rows
    bias = dev(torch.randn(E, generator=g) * 0.1)
    for b in (None, bias):
        for top2 in (False, True):
            for renorm in (False, True):
                check(l, b, k, kind, groups, topg, top2, renorm, 2.5)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_and_infinite_logits(kind, groups):
    g = torch.Generator().manual_seed(5)
    T, E, k = 12, 64, 6
    l = torch.randn(T, E, generator=g)
    l[0] = -np.inf                       # nothing left
    l[1, 1:] = -np.inf                   # one expert left
    l[2, :5] = -np.inf
    l[3] = torch.finfo(torch.float32).min
    l[4, ::2] = torch.finfo(torch.float32).min
    l[5, 7] = np.inf
    l[6, 3] = np.nan
    l[7] = np.nan
    l[8, 16:] = -np.inf                  # whole groups masked
    l[9, 17], l[9, 40] = -np.inf, np.nan
    l[10] = 0.0
    l[10, ::3] = -0.0                    # ties of both zeros
    bias = torch.randn(E, generator=g) * 0.1
    odd = bias.clone()
    odd[3], odd[9], odd[30] = -np.inf, np.nan, np.inf
    for b in (None, bias, odd):
        for top2 in (False, True):
            for renorm in (False, True):
                check(dev(l), None if b is None else dev(b), k, kind, groups, min(groups, 2), top2, renorm)


def test_equal_logits_go_to_the_lower_expert():
    l = torch.zeros(3, 320, device="cuda")
    l[1, 200:] = 1.0
    for bias in (None, torch.zeros(320, device="cuda")):
        for groups, topg in ((1, 1), (8, 2)):
            for kind in KIND:
                check(l, bias, 8, kind, groups, topg, True)


def test_sums_nearer_than_32_bits():
    """Logits and biases whose sums of score and bias are equal up to 2^-30 or so: 64 bits decide."""
    rng = np.random.default_rng(0)
    T, E, k = 200, 96, 8
    l = rng.normal(size=(T, E)).astype(np.float32)
    # the bias of an expert makes up for its score in token 0; the other tokens' logits differ by ulps
    for kind in KIND:
        s = np.array([ref.scores(l[0].astype(np.float64), kind)])[0]
        bias = (0.9 - s).astype(np.float32)
        near = l[0] * (1 + rng.integers(-2, 3, size=(T, E)) * 2.0 ** -23)
        check(dev(near.astype(np.float32)), dev(bias), k, kind)
        check(dev(near.astype(np.float32)), dev(bias), k, kind, 8, 3, True, False)


@pytest.mark.parametrize("biased", [False, True])
def test_groups_nearer_than_32_bits(biased):
    """Groups whose two largest scores (or whose largest score and bias) have sums that are equal up to
    2^-24 or so."""
    rng = np.random.default_rng(1)
    T, G, n = 300, 8, 20
    for kind, mid in (("softmax", 0.5), ("sigmoid", 0.5), ("sigmoid", 0.55)):
        l = rng.uniform(-9, -6, size=(T, G, n))
        d = rng.uniform(0.01, 0.3, size=(T, G))
        for i, v in enumerate((mid + d, mid - d)):
            at = np.log(v / (1 - v)) if kind == "sigmoid" else np.log(v)
            np.put_along_axis(l, np.full((T, G, 1), 3 + 5 * i), at[..., None], 2)
        l = l.reshape(T, G * n).astype(np.float32)
        bias = None
        if biased:   # of one expert a group, by which the largest keys of token 0 are equal
            s = np.stack([ref.scores(r, kind) for r in l.astype(np.float64)]).reshape(T, G, n)
            bias = np.zeros((G, n))
            bias[:, 3] = 2 - s[0, :, 3]
            l[1:, 3::n] = l[0, 3::n] + rng.integers(-2, 3, size=(T - 1, G)) * 2.0 ** -24
            if kind == "softmax":   # the same sum of exponentials for every token, or nearly
                l[1:] = np.where(np.isin(np.arange(G * n) % n, (3,)), l[1:], l[0])
            bias = dev(bias.reshape(-1))
        for topg in (1, 3, 7):
            if kind == "sigmoid" and mid == 0.5 and not biased:
                # the two logits are each other's negatives, their scores' sums 1 and their order that of
                # 64-bit roundings: any groups, but the largest in the ones chosen
                ids, _ = run(dev(l), bias, 2, kind, G, topg, True, False)
                assert torch.all((ids % n == 3) | (ids % n == 8))
                continue
            check(dev(l), bias, 2, kind, G, topg, not biased, False)


def test_far_logits():
    """Scores that are 0 or 1 in 32 bits: renormalised weights are still their quotients."""
    l = torch.tensor([[-120.0, -121.0, -125.0, -300.0], [-30.0, -31.0, 40.0, 41.0], [90.0, 95.0, -95.0, 20.0],
                      [-3e38, -3e38, -3e38, -3e38]], device="cuda")
    for kind in KIND:
        check(l, None, 3, kind)
        check(l[:2], None, 3, kind, renorm=False)


def test_no_tokens_and_other_streams():
    ids, w = run(torch.empty(0, 8, device="cuda"), None, 2, "softmax")
    assert ids.shape == (0, 2)
    l = torch.randn(50, 320, device="cuda")
    want = run(l, None, 8, "softmax")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(l, None, 8, "softmax")
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    got = run(l, None, 8, "softmax", stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_in_a_graph():
    l = torch.randn(70, 64, device="cuda")
    ids, w = torch.empty(70, 4, dtype=torch.int32, device="cuda"), torch.empty(70, 4, device="cuda")
    dl = torch.empty_like(l)
    bias = torch.randn(64, device="cuda") * 0.1

    def step():
        moe.moe_route_scores(l, ids, w, bias=bias, score=moe.MOE_SCORE_SIGMOID, num_groups=4, topk_groups=2)
        moe.moe_route_scores_backward(l, ids, w, dl, score=moe.MOE_SCORE_SIGMOID)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        l.copy_(torch.randn_like(l))
        step()
        want = ids.clone(), w.clone(), dl.clone()
        ids.zero_(), w.zero_(), dl.zero_()
        graph.replay()
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1]) and torch.equal(dl, want[2])


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 8), (70, 320, 8), (33, 1000, 32), (9, 61, 3)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_gradient(T, E, k, kind, renorm, dtype):
    g = torch.Generator().manual_seed(E + k)
    l = dev(torch.randn(T, E + 5, generator=g) * 2, DT[dtype])[:, :E]
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    dw = torch.randn(T, k, generator=g)
    out = torch.full((T, E + 1), -7.0, device="cuda").to(DT[dtype])
    moe.moe_route_scores_backward(l, ids.cuda(), dw.cuda(), out[:, :E], score=KIND[kind], renormalise=renorm,
                                  scale=2.5)
    l64, d64 = l.double().cpu().numpy(), dw.double().numpy()
    want = ref.route_grad(l64, ids.numpy(), d64, kind, renorm, 2.5)
    got = out[:, :E].double().cpu().numpy()
    # a product of scores (W_TOL each) and a difference of terms of at most sum |g| p, rounded once
    mag = np.abs(d64).max(1, keepdims=True) * 2.5
    s = np.stack([ref.scores(r, kind) for r in l64])
    if renorm:
        s = np.ones_like(s)
    bound = 3 * W_TOL * mag * (s + 1e-30) * k + UNIT[dtype] * np.abs(want) + 2.0 ** -24 * (dtype == "fp16") + 1e-38
    assert np.all(np.abs(got - want) <= bound)
    assert torch.all(out[:, E] == -7)


def test_gradient_against_differences():
    rng = np.random.default_rng(2)
    T, E, k = 2, 12, 4
    l = rng.normal(size=(T, E)).astype(np.float32).astype(np.float64)
    dw = rng.normal(size=(T, k))
    for kind in KIND:
        for renorm in (False, True):
            ids, _ = ref.route(l, None, k, kind, 1, 1, False, renorm, 1.5)

            def loss(x):
                out = 0.0
                for t in range(T):
                    w = ref.scores(x[t], kind)[ids[t]]
                    out += (dw[t] * 1.5 * (w / w.sum() if renorm else w)).sum()
                return out

            num = np.zeros_like(l)
            for i in np.ndindex(l.shape):
                d = np.zeros_like(l)
                d[i] = 1e-5
                num[i] = (loss(l + d) - loss(l - d)) / 2e-5
            out = torch.empty(T, E, device="cuda")
            moe.moe_route_scores_backward(dev(l), dev(ids, torch.int32), dev(dw), out, score=KIND[kind],
                                          renormalise=renorm, scale=1.5)
            # central differences are off by h^2 and 2^-53 / h; the gradient by some 2^-20 of its terms
            assert np.abs(out.double().cpu().numpy() - num).max() < 1e-5


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_gradient_where_one_weight_is_nearly_all(kind):
    """Renormalised weights of 1 - 1e-7 and 1e-7: the differences of their gradients, not what is left of
    them."""
    l = torch.tensor([[16.0, -0.1, 0.3, 1.0], [-2.0, -18.0, -19.0, -17.5]], device="cuda")
    ids = torch.tensor([[0, 1, 2], [0, 1, 3]], dtype=torch.int32, device="cuda")
    dw = torch.tensor([[0.9, -0.4, 0.3], [-1.0, 0.7, 0.2]], device="cuda")
    out = torch.empty_like(l)
    moe.moe_route_scores_backward(l, ids, dw, out, score=KIND[kind])
    want = ref.route_grad(l.double().cpu().numpy(), ids.cpu().numpy(), dw.double().cpu().numpy(), kind, True, 1.0)
    # each term within W_TOL of itself; of a sigmoid 1 - s is one more (1 / (1 + e^l), 2^-22)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 3 * (W_TOL + 2.0 ** -22) * np.abs(dw.double().cpu().numpy()).max() *
                  np.maximum(np.abs(want) / 0.5, 1e-12))


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_the_same_expert_twice_and_of_ids_out_of_range(kind, renorm):
    rng = np.random.default_rng(3)
    l = rng.normal(size=(4, 10)).astype(np.float32).astype(np.float64)
    l[3, 2:6] = -np.inf
    ids = np.array([[1, 1, 3], [2, -1, 10], [5, 2000000000, -2000000000], [2, 3, 7]])
    dw = rng.normal(size=(4, 3)).astype(np.float32).astype(np.float64)
    out = torch.empty(4, 10, device="cuda")
    moe.moe_route_scores_backward(dev(l), dev(ids, torch.int32), dev(dw), out, score=KIND[kind],
                                  renormalise=renorm)
    want = ref.route_grad(l, ids, dw, kind, renorm, 1.0)
    assert np.abs(out.double().cpu().numpy() - want).max() <= 9 * W_TOL * np.abs(dw).max()


def test_gradient_of_masked_tokens():
    l = torch.full((3, 16), -np.inf, device="cuda")
    l[1, 4] = 1.0
    l[2, 3] = np.nan
    ids = torch.tensor([[0, 1], [4, 0], [1, 3]], dtype=torch.int32, device="cuda")
    dw = torch.ones(3, 2, device="cuda")
    for kind in KIND.values():
        for renorm in (False, True):
            out = torch.empty(3, 16, device="cuda")
            moe.moe_route_scores_backward(l, ids, dw, out, score=kind, renormalise=renorm)
            assert torch.all(out[0] == 0) and torch.isfinite(out[1]).all() and torch.isnan(out[2, 3])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_a_token_with_nan_weights_has_nan_gradients(kind, renorm, dtype):
    """Whichever logit it is: one that is not chosen, too."""
    T, E, k = 5, 70, 4
    g = torch.Generator("cuda").manual_seed(8)
    l = torch.randn(T, E, generator=g, device="cuda").to(dtype)
    l[1, 69] = float("nan")
    l[2, 3] = float("inf")
    l[3, 40] = -float("inf")
    bias = torch.zeros(E, device="cuda")
    bias[3] = -float("inf")   # (the infinite logit is not chosen)
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    how = dict(score=KIND[kind], renormalise=renorm)
    moe.moe_route_scores(l, ids, w, bias=bias, **how)
    assert not torch.any(ids[1] == 69) and not torch.any(ids[2] == 3)
    d = torch.empty_like(l)
    moe.moe_route_scores_backward(l, ids, torch.randn(T, k, generator=g, device="cuda"), d, **how)
    bad = [False, True, kind == "softmax", False, False]
    for t in range(T):
        assert bool(torch.isnan(w[t]).all()) == bad[t] == bool(torch.isnan(w[t]).any())
        assert bool(torch.isnan(d[t]).all()) == bad[t] == bool(torch.isnan(d[t]).any())


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 2])
def test_equal_keys_at_the_border_below_a_near_one(kind, groups):
    """Each token has three experts, the others are masked: a first one whose key lies within a rounding
    of two equal ones.  Of k = 2 the pair is chosen where it is larger, else the first and the lower one."""
    T, k = 300, 2
    rng = np.random.default_rng(groups)
    E = 1024
    l = np.full((T, E), -np.inf, np.float32)
    bias = rng.normal(size=E).astype(np.float32)
    a = 3 * np.arange(T) + 1
    row = np.arange(T)
    la, lb = rng.normal(size=(2, T)).astype(np.float32)
    l[row, a], l[row, a + 1], l[row, a + 2] = la, lb, lb
    bias[a + 2] = bias[a + 1]
    sa, sb = (1 / (1 + np.exp(-x.astype(np.float64))) for x in (la, lb))
    if kind == "softmax":
        ea, eb = np.exp(la.astype(np.float64)), np.exp(lb.astype(np.float64))
        sa, sb = ea / (ea + 2 * eb), eb / (ea + 2 * eb)
    bias[a] = sb + bias[a + 1].astype(np.float64) - sa     # (rounded: the keys differ by that)
    first = sa + bias[a] > sb + bias[a + 1]
    assert 100 < first.sum() < 200
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_route_scores(torch.from_numpy(l).cuda(), ids, w, bias=torch.from_numpy(bias).cuda(), score=KIND[kind],
                         num_groups=groups, topk_groups=groups)
    want = np.where(first[:, None], np.stack([a, a + 1], 1), np.stack([a + 1, a + 2], 1))
    assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("k,groups,topg", [(1, 1, 1), (2, 1, 1), (3, 1, 1), (1, 32, 1), (2, 32, 2), (40 // 8, 32, 2)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_keys_near_by_every_measure(kind, k, groups, topg):
    """Each token has two experts far above the others, in two groups, with keys from 2^-29 to 2^-14 apart."""
    rng = np.random.default_rng(k + groups)
    T, E = 500, 1024
    a, row = np.arange(T), np.arange(T)
    b = a + 512
    l = rng.normal(size=(T, E)).astype(np.float32) - 8
    l[row, a], l[row, b] = 1 + 0.1 * rng.normal(size=(2, T))
    e = np.exp(l.astype(np.float64))
    s = e / e.sum(1, keepdims=True) if kind == "softmax" else 1 / (1 + np.exp(-l.astype(np.float64)))
    apart = 2.0 ** rng.uniform(-29, -14, size=T) * rng.choice([-1, 1], size=T)
    bias = np.zeros(E, np.float32)
    bias[a] = s[row, b] - s[row, a] + apart
    assert 100 < (s[row, a] + bias[a] > s[row, b] + bias[b]).sum() < 400
    check(dev(l), dev(bias), k, kind, groups, topg)


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_equal_keys_at_the_border_and_larger_ones_behind(dtype):
    """Experts of equal terms before others whose keys differ from theirs in 64 bits alone."""
    l = torch.tensor([[-34.5, 22.75, -37.25, -5.25, -5.0, -31.5, 22.75, 31.75, 84.25],
                      [22.75, 22.75, 22.75, 22.75, 22.75, 22.75, 22.75, 22.75, 24.0],
                      [22.75] * 9, [0.0] * 9])
    for bias in (torch.zeros(9), torch.full((9,), 0.25)):
        for k in range(1, 9):
            check(dev(l, DT[dtype]), dev(bias), k, "sigmoid")
    many = torch.full((3, 400), 22.75)
    many[0, 399] = 30.0
    many[1, 200:] = 23.0
    for k in (1, 8, 31, 32):
        check(dev(many, DT[dtype]), dev(torch.zeros(400)), k, "sigmoid")
