"""Plain 64-bit implementations of the handle-free operators: the sort of routed pairs, dispatch,
combine and their gradients, MXFP4 quantisation and the grouped product (numpy only)."""
import numpy as np

E2M1_MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])

# unit roundoff of a rounding to the type (to nearest), and its smallest subnormal step
UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
STEP = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24, "fp32": 2.0 ** -149}


def sort_pairs(ids, E, off, El, align, cap):
    """ids [T, k] -> counts, offsets, perm_src, inv, bad id seen, overflow seen."""
    flat = np.asarray(ids).reshape(-1)
    groups = [[] for _ in range(El)]
    bad = False
    for p, e in enumerate(flat):
        if e < 0 or e >= E:
            bad = True
        elif 0 <= e - off < El:
            groups[e - off].append(p)
    counts = np.array([len(g) for g in groups], np.int32).reshape(El)
    offsets = np.zeros(El + 1, np.int32)
    for e in range(El):
        offsets[e + 1] = offsets[e] + (len(groups[e]) + align - 1) // align * align
    perm = np.full(cap, -1, np.int32)
    inv = np.full(flat.size, -1, np.int32)
    over = False
    for e, g in enumerate(groups):
        for i, p in enumerate(g):
            r = int(offsets[e]) + i
            if r < cap:
                perm[r], inv[p] = p, r
            else:
                over = True
    return counts, offsets, perm, inv, bad, over


def gather_sum(rows, inv, w, T, k):
    """(sum_j w rows[inv], sum_j |w rows[inv]|) in fp64; w None: ones."""
    H = rows.shape[1]
    out, mag = np.zeros((T, H)), np.zeros((T, H))
    inv = inv.reshape(T, k)
    for j in range(k):
        t = np.flatnonzero((inv[:, j] >= 0) & (inv[:, j] < rows.shape[0]))
        v = rows[inv[t, j]] * (1.0 if w is None else w[t, j][:, None].astype(np.float64))
        out[t] += v
        mag[t] += np.abs(v)
    return out, mag


def rounded_ok(got, ref, slack, kind):
    """|got - ref| within `slack` (the error before the last rounding) and one rounding to `kind`."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    both_nan = np.isnan(got) & np.isnan(ref)
    u = UNIT[kind]
    return both_nan | (np.abs(got - ref) <= u * (np.abs(ref) + slack) + slack + STEP[kind])


def quant_mxfp4(x, ceil):
    """x [R, K] fp64 (values of the input type) -> codes 0..15 [R, K], scale bytes [R, K / 32],
    values [R, K] fp64."""
    R, K = x.shape
    b = np.asarray(x, np.float64).reshape(-1, 32)
    good = np.all(np.isfinite(b), axis=1)
    m = np.max(np.abs(np.where(good[:, None], b, 0.0)), axis=1)
    e = np.frexp(m)[1].astype(np.int64) - 1 - 2            # m = f 2^(e + 3), f in [1/2, 1)
    if ceil:
        e += m > 6 * np.ldexp(1.0, e)
    e = np.where(m == 0, -127, np.clip(e, -127, 127))
    q = np.ldexp(np.abs(np.where(good[:, None], b, 0.0)), -e[:, None])
    # the nearest value; of two as near (neighbouring codes) the even code
    d = np.abs(q[..., None] - E2M1_MAG)
    best = d == d.min(-1, keepdims=True)
    even = best & (np.arange(8) % 2 == 0)
    c = np.where(even.any(-1), even.argmax(-1), best.argmax(-1))
    vals = np.ldexp(np.copysign(E2M1_MAG[c], b), e[:, None])
    codes = np.where(good[:, None], c + 8 * np.signbit(b), 0)
    vals[~good] = np.nan
    sf = np.where(good, e + 127, 255)
    return codes.reshape(R, K), sf.reshape(R, K // 32), vals.reshape(R, K)


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    p = np.asarray(packed).astype(np.int64)
    return np.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], -1)


def tile_scales(sf, fill=0):
    """[R, K / 32] -> the tiled layout, rows past R filled."""
    R, S = sf.shape
    RB, KA = (R + 127) // 128, (S + 3) // 4
    out = np.full(RB * KA * 512, fill, np.uint8)
    r, kb = np.arange(R)[:, None], np.arange(KA * 4)[None, :]
    at = ((r >> 7) * KA + (kb >> 2)) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + kb % 4
    out[at] = np.pad(np.asarray(sf), ((0, 0), (0, KA * 4 - S)))
    return out


def decode(codes, sf):
    """codes 0..15 [R, K], scale bytes [R, K / 32] -> fp64."""
    v = np.where(codes >= 8, -1.0, 1.0) * E2M1_MAG[codes & 7]
    s = np.where(sf == 255, np.nan, 2.0 ** (np.minimum(sf, 254).astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1)
