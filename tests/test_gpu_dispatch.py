"""Dispatch, weighted combine and their gradients against plain 64-bit implementations.

Tolerances: a sum of n terms in fp32 (any order, fused or not) is within n 2^-23 of the sum of
the terms' magnitudes; then one rounding to the output's type."""
import numpy as np
import pytest
import torch

import nvfp4_mixture_experts_gb300 as moe
import ops_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F = 2.0 ** -23


def f64(t):
    return t.detach().cpu().double().numpy()


def make_ids(rng, T, E, k, kind):
    if kind == "one":
        return np.full((T, k), E - 1, np.int32)
    if kind == "skewed":
        return np.minimum(rng.geometric(0.3, (T, k)) - 1, E - 1).astype(np.int32)
    if T == 0:
        return np.zeros((0, k), np.int32)
    return np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)


def run_dispatch(x, ids, E, off, El, align, cap, H=0, stream=None):
    T, k = ids.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    o = dict(counts=torch.full((El,), -7, **i32), offsets=torch.full((El + 1,), -7, **i32),
             perm=torch.full((cap,), -7, **i32), inv=torch.full((T * k,), -7, **i32),
             status=torch.zeros(1, **i32), rows=None)
    if x is not None:
        o["rows"] = torch.full((cap, x.shape[1]), -3.0, dtype=x.dtype, device="cuda")
    moe.moe_dispatch(x, torch.from_numpy(ids).cuda(), E, off, El, align, o["counts"],
                     o["offsets"], o["perm"], o["inv"], o["rows"], o["status"], stream)
    torch.cuda.synchronize()
    return o


SORTS = [  # T, E, k, off, El, align, kind
    (1, 1, 1, 0, 1, 1, "spread"), (1, 320, 8, 0, 320, 128, "spread"),
    (1, 320, 8, 319, 1, 128, "spread"), (3, 8, 8, 2, 0, 16, "spread"),
    (17, 5, 3, 1, 3, 4, "spread"), (64, 320, 8, 160, 160, 128, "spread"),
    (128, 16, 8, 0, 16, 128, "one"), (129, 16, 8, 0, 16, 1, "skewed"),
    (1000, 60, 5, 11, 37, 1, "spread"), (2048, 1024, 2, 0, 1024, 128, "spread"),
    (777, 40, 32, 3, 30, 2, "spread"), (5000, 320, 8, 0, 320, 1, "skewed"),
    (1025, 4, 1, 0, 4, 128, "one"), (0, 4, 2, 0, 4, 8, "spread"),
]


@pytest.mark.parametrize("T,E,k,off,El,align,kind", SORTS)
def test_maps_are_the_stable_sort(T, E, k, off, El, align, kind):
    ids = make_ids(np.random.default_rng(T + E), T, E, k, kind)
    cap = moe.moe_dispatch_rows_capacity(T, k, El, align)
    o = run_dispatch(None, ids, E, off, El, align, cap)
    counts, offsets, perm, inv, _, over = ref.sort_pairs(ids, E, off, El, align, cap)
    assert not over
    assert np.array_equal(o["counts"].cpu(), counts)
    assert np.array_equal(o["offsets"].cpu(), offsets)
    assert np.array_equal(o["perm"].cpu(), perm)
    assert np.array_equal(o["inv"].cpu(), inv)
    assert o["status"].item() == 0


@pytest.mark.parametrize("T", [20, 700])
def test_bad_ids_are_dropped_and_flagged(T):
    ids = make_ids(np.random.default_rng(1), T, 12, 3, "spread")
    ids[3, 1], ids[7, 0], ids[T - 1, 2] = -1, 12, 2 ** 30
    cap = moe.moe_dispatch_rows_capacity(T, 3, 12, 8)
    x = torch.randn(T, 40, device="cuda")
    o = run_dispatch(x, ids, 12, 0, 12, 8, cap)
    counts, offsets, perm, inv, bad, _ = ref.sort_pairs(ids, 12, 0, 12, 8, cap)
    assert bad and o["status"].item() == moe.MOE_DEV_BAD_EXPERT_ID
    assert np.array_equal(o["perm"].cpu(), perm) and np.array_equal(o["inv"].cpu(), inv)
    assert np.array_equal(o["counts"].cpu(), counts)


@pytest.mark.parametrize("T,cap", [(20, 37), (700, 1000), (20, 1)])
def test_rows_past_the_capacity_are_dropped_and_flagged(T, cap):
    ids = make_ids(np.random.default_rng(2), T, 12, 3, "spread")
    x = torch.randn(T, 40, device="cuda")
    o = run_dispatch(x, ids, 12, 0, 12, 8, cap)
    counts, offsets, perm, inv, _, over = ref.sort_pairs(ids, 12, 0, 12, 8, cap)
    assert over and o["status"].item() == moe.MOE_DEV_ROWS_OVERFLOW
    assert np.array_equal(o["perm"].cpu(), perm) and np.array_equal(o["inv"].cpu(), inv)
    assert np.array_equal(o["counts"].cpu(), counts)
    live = perm >= 0
    assert np.array_equal(f64(o["rows"])[live], f64(x)[perm[live] // 3])


def test_padding_alone_past_the_capacity_is_no_overflow():
    ids = np.zeros((3, 1), np.int32)
    o = run_dispatch(None, ids, 2, 0, 2, 128, 3)
    assert o["status"].item() == 0 and o["perm"].tolist() == [0, 1, 2]


ROWS = [  # T, H, E, k, off, El, align, ld, shift
    (1, 4096, 320, 8, 0, 320, 128, 0, 0), (1, 1, 4, 2, 0, 4, 1, 0, 0),
    (33, 1001, 20, 5, 3, 9, 1, 6, 0), (64, 256, 16, 2, 0, 16, 128, 24, 0),
    (64, 256, 16, 2, 0, 16, 128, 3, 0), (50, 520, 9, 9, 2, 2, 16, 8, 1),
    (300, 136, 32, 8, 0, 32, 4, 0, 0), (7, 2055, 40, 32, 0, 40, 1, 1, 0),
    (40, 64, 8, 8, 4, 0, 1, 0, 0), (200, 4104, 64, 4, 0, 64, 1, 0, 0),
    # rows shorter than a piece, and every distance of rows from 16 bytes
    (70, 3, 6, 2, 0, 6, 1, 0, 0), (9, 7, 6, 2, 0, 6, 2, 2, 1), (600, 5, 6, 2, 1, 4, 1, 0, 3),
    (40, 4001, 16, 2, 0, 16, 1, 0, 0), (300, 1026, 16, 4, 0, 16, 1, 2, 0),
    (130, 2300, 16, 8, 0, 16, 1, 0, 2), (20, 777, 12, 12, 0, 12, 1, 9, 5),
    # one or two pairs a token, several tokens together, the last ones fewer
    (259, 4104, 16, 1, 0, 16, 1, 0, 0), (403, 1001, 20, 2, 3, 9, 1, 6, 0),
    (1031, 520, 9, 1, 2, 4, 16, 8, 1), (258, 2300, 16, 2, 0, 16, 1, 2, 2),
    (3001, 136, 8, 2, 4, 2, 1, 0, 0), (301, 7, 5, 1, 0, 5, 1, 1, 0),
    (2501, 264, 6, 1, 0, 6, 128, 0, 0), (256, 2048, 4, 2, 0, 4, 1, 4, 0),
]


def token_rows(T, H, ld, shift, dtype, seed, nan=False):
    """[T, H] with row stride H + ld, starting `shift` elements into its storage."""
    g = torch.Generator().manual_seed(seed)
    n = T * (H + ld) + shift
    flat = torch.full((n,), float("nan")) if nan else torch.randn(n, generator=g)
    return flat.to(dtype).cuda()[shift:].view(T, H + ld)[:, :H]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,E,k,off,El,align,ld,shift", ROWS)
def test_rows_and_their_way_back(T, H, E, k, off, El, align, ld, shift, dtype):
    dt, rng = DT[dtype], np.random.default_rng(T * H)
    ids = make_ids(rng, T, E, k, "spread")
    cap = moe.moe_dispatch_rows_capacity(T, k, El, align)
    x = token_rows(T, H, ld, shift, dt, 5)
    o = run_dispatch(x, ids, E, off, El, align, cap)
    _, _, perm, inv, _, _ = ref.sort_pairs(ids, E, off, El, align, cap)
    live = perm >= 0
    got = f64(o["rows"])
    assert np.array_equal(got[live], f64(x)[perm[live] // k])
    assert np.all(got[~live] == -3.0), "rows of no pair are left as they are"

    # rows of no pair hold NaN: none of it may reach a result
    y = torch.randn(cap, H).to(dt).cuda()
    y[torch.from_numpy(~live).cuda()] = float("nan")
    w = torch.rand(T, k, device="cuda") + 0.1
    w[torch.from_numpy(inv.reshape(T, k) < 0).cuda()] = float("nan")
    for weight in (None, w):
        out = token_rows(T, H, ld, shift, dt, 6, nan=True)
        if weight is None:
            moe.moe_dispatch_backward(y, o["inv"], k, out)
        else:
            moe.moe_combine_weighted(y, o["inv"], weight, out)
        want, mag = ref.gather_sum(f64(y), inv, None if weight is None else f64(w), T, k)
        ok = ref.rounded_ok(f64(out), want, (k + 1) * F * mag, dtype)
        assert np.all(ok)

    dout = token_rows(T, H, ld, shift, dt, 7)
    dy = torch.full((cap, H), -3.0, dtype=dt, device="cuda")
    dw = torch.full((T, k), -3.0, device="cuda")
    moe.moe_combine_backward(dout, y, o["inv"], w, dy, dw)
    d, yy, ww = f64(dout), f64(y), f64(w)
    got_dy, got_dw = f64(dy), f64(dw)
    assert np.all(got_dy[~live] == -3.0)
    t, j = perm[live] // k, perm[live] % k
    want = d[t] * ww[t, j][:, None]
    assert np.all(ref.rounded_ok(got_dy[live], want, F * np.abs(want), dtype))
    terms = d[t] * yy[live]
    assert np.all(np.abs(got_dw[t, j] - terms.sum(1)) <= (H + 2) * F * np.abs(terms).sum(1) + 1e-40)
    dropped = inv.reshape(T, k) < 0
    assert np.all(got_dw[dropped] == 0.0)

    # one gradient at a time gives the same numbers
    dy2, dw2 = torch.full_like(dy, -3.0), torch.full_like(dw, -3.0)
    moe.moe_combine_backward(dout, y, o["inv"], w, None, dw2)
    moe.moe_combine_backward(dout, None, o["inv"], w, dy2, None)
    assert torch.equal(dy2, dy) and torch.equal(dw2, dw)


def test_gradients_are_the_differences():
    """The operators are linear in x, y and w one at a time, so a difference quotient with step 1
    is the directional derivative up to fp32 rounding."""
    T, H, E, k, El, off = 37, 200, 16, 4, 11, 3
    rng = np.random.default_rng(3)
    ids = make_ids(rng, T, E, k, "spread")
    cap = moe.moe_dispatch_rows_capacity(T, k, El, 8)
    x, vx = torch.randn(T, H, device="cuda"), torch.randn(T, H, device="cuda")
    o = run_dispatch(x, ids, E, off, El, 8, cap)
    live = (o["perm"] >= 0)[:, None]
    g = torch.randn(cap, H, device="cuda")
    up = run_dispatch(x + vx, ids, E, off, El, 8, cap)["rows"]
    down = run_dispatch(x - vx, ids, E, off, El, 8, cap)["rows"]
    diff = float((torch.where(live, (up.double() - down.double()) / 2 * g.double(), 0.0)).sum())
    dx = torch.empty_like(x)
    moe.moe_dispatch_backward(g, o["inv"], k, dx)
    mag = float((dx.abs().double() * vx.abs().double()).sum()) + float((g[live[:, 0]].abs()).sum()) * 8
    assert abs(float((dx.double() * vx.double()).sum()) - diff) <= (k + 4) * F * mag

    y, vy = torch.randn(cap, H, device="cuda"), torch.randn(cap, H, device="cuda")
    w, vw = torch.rand(T, k, device="cuda"), torch.randn(T, k, device="cuda")
    dout = torch.randn(T, H, device="cuda")

    def loss(y, w):
        out = torch.empty(T, H, device="cuda")
        moe.moe_combine_weighted(y, o["inv"], w, out)
        return float((out.double() * dout.double()).sum())

    dy, dw = torch.zeros_like(y), torch.empty_like(w)
    moe.moe_combine_backward(dout, y, o["inv"], w, dy, dw)
    mag = float((dout.abs().double().sum(0) * 1.0).sum()) * k * 16
    for a, b, grad in (((y + vy, w), (y - vy, w), float((dy.double() * vy.double()).sum())),
                       ((y, w + vw), (y, w - vw), float((dw.double() * vw.double()).sum()))):
        assert abs((loss(*a) - loss(*b)) / 2 - grad) <= (H + k) * F * mag


def test_infinities_and_nans_of_live_rows_stay_in_their_token():
    T, H, E, k = 12, 64, 6, 2
    ids = make_ids(np.random.default_rng(8), T, E, k, "spread")
    o = run_dispatch(None, ids, E, 0, E, 1, T * k)
    inv = o["inv"].cpu().numpy().reshape(T, k)
    y = torch.randn(T * k, H, device="cuda")
    y[inv[3, 0], 5], y[inv[4, 1], 6] = float("inf"), float("nan")
    w = torch.rand(T, k, device="cuda")
    w[3, 0] = 0.0   # zero times infinity is NaN by the formula
    out = torch.empty(T, H, device="cuda")
    moe.moe_combine_weighted(y, o["inv"], w, out)
    bad = ~torch.isfinite(out).cpu().numpy()
    assert np.argwhere(bad).tolist() == [[3, 5], [4, 6]]


def test_another_stream_orders_the_calls():
    T, H, E, k = 512, 1024, 32, 4
    ids = make_ids(np.random.default_rng(9), T, E, k, "spread")
    cap = moe.moe_dispatch_rows_capacity(T, k, E, 1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x = torch.zeros(T, H, device="cuda")
        for _ in range(20):
            x += 1.0                      # the calls below must see the last addition
        o = run_dispatch_async(x, ids, E, cap)
        dx = torch.empty(T, H, device="cuda")
        moe.moe_dispatch_backward(o[1], o[0], k, dx)
    side.synchronize()
    assert torch.all(dx == 20.0 * k)


def run_dispatch_async(x, ids, E, cap):
    i32 = dict(dtype=torch.int32, device="cuda")
    T, k = ids.shape
    inv, rows = torch.empty(T * k, **i32), torch.empty(cap, x.shape[1], device="cuda")
    moe.moe_dispatch(x, torch.from_numpy(ids).cuda(), E, 0, E, 1, torch.empty(E, **i32),
                     torch.empty(E + 1, **i32), torch.empty(cap, **i32), inv, rows)
    return inv, rows


def test_indices_out_of_range_count_as_dropped():
    T, H, k, cap = 6, 48, 2, 9
    inv = torch.tensor([0, 1, -1, 9, 2 ** 30, -5, 3, 3, 8, 7, -1, -1], dtype=torch.int32).cuda()
    y, w = torch.randn(cap, H, device="cuda"), torch.rand(T, k, device="cuda")
    out = torch.empty(T, H, device="cuda")
    moe.moe_combine_weighted(y, inv, w, out)
    want, mag = ref.gather_sum(f64(y), inv.cpu().numpy(), f64(w), T, k)
    assert np.all(ref.rounded_ok(f64(out), want, 3 * F * mag, "fp32"))
    dw = torch.full((T, k), -3.0, device="cuda")
    moe.moe_combine_backward(out, y, inv, w, None, dw)
    assert dw.view(-1)[[2, 3, 4, 5, 10, 11]].abs().sum() == 0


def test_rows_past_two_to_the_31_bytes():
    """A row buffer of over 2^32 elements: the row offsets need 64 bits."""
    H, cap = 4096, (1 << 20) + 64
    y = torch.zeros(cap, H, dtype=torch.bfloat16, device="cuda")
    y[cap - 1], y[cap - 2] = 3.0, 5.0
    inv = torch.tensor([cap - 1, cap - 2], dtype=torch.int32).cuda()
    w = torch.tensor([[2.0, 1.0]], device="cuda")
    out = torch.empty(1, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_combine_weighted(y, inv, w, out)
    assert torch.all(out == 11.0)
    dy, dw = y, torch.empty(1, 2, device="cuda")
    moe.moe_combine_backward(out, None, inv, w, dy, None)
    assert torch.all(dy[cap - 1] == 22.0) and torch.all(dy[cap - 2] == 11.0)
    assert torch.all(dy[cap - 3] == 0.0)


@pytest.mark.parametrize("T", [40, 900])
def test_calls_replay_in_a_graph(T):
    """Captured dispatch (both launch forms), combine and gradient follow new ids and inputs."""
    E, k, H = 24, 3, 96
    rng = np.random.default_rng(T)
    ids = torch.from_numpy(make_ids(rng, T, E, k, "spread")).cuda()
    x, w = torch.randn(T, H, device="cuda"), torch.rand(T, k, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets, perm = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T * k, **i32)
    inv, rows = torch.empty(T * k, **i32), torch.empty(T * k, H, device="cuda")
    out, dy, dw = torch.empty(T, H, device="cuda"), torch.empty(T * k, H, device="cuda"), torch.empty(T, k, device="cuda")

    def step():
        moe.moe_dispatch(x, ids, E, 0, E, 1, counts, offsets, perm, inv, rows)
        moe.moe_combine_weighted(rows, inv, w, out)
        moe.moe_combine_backward(out, rows, inv, w, dy, dw)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    new = make_ids(rng, T, E, k, "spread")
    ids.copy_(torch.from_numpy(new))
    x.copy_(torch.randn(T, H))
    g.replay()
    torch.cuda.synchronize()
    _, _, want_perm, want_inv, _, _ = ref.sort_pairs(new, E, 0, E, 1, T * k)
    assert np.array_equal(perm.cpu(), want_perm) and np.array_equal(inv.cpu(), want_inv)
    assert np.array_equal(f64(rows), f64(x)[want_perm // k])
    want, mag = ref.gather_sum(f64(rows), want_inv, f64(w), T, k)
    assert np.all(ref.rounded_ok(f64(out), want, (k + 1) * F * mag, "fp32"))
    d = f64(out)[want_perm // k] * f64(rows)
    got = f64(dw).reshape(-1)[want_perm]
    assert np.all(np.abs(got - d.sum(1)) <= (H + 2) * F * np.abs(d).sum(1))
