"""Plain 64-bit implementations of the operators around the experts: routing from logits, the
root-mean-square norm, MXFP8 quantisation and the gate, with their gradients (numpy only)."""
import numpy as np

# the E4M3 numbers by code 0..126 (127 is NaN): subnormals m 2^-9, then (8 + m) 2^(e - 10)
_C = np.arange(127)
E4M3_MAG = np.where(_C < 8, _C * 2.0 ** -9, (8 + _C % 8) * 2.0 ** (_C // 8 - 10.0))


def e4m3_codes(q):
    """Codes of |q| (finite): the nearest number, of two as near the even code, at most 448."""
    q = np.minimum(np.abs(q), 448.0)
    hi = np.clip(np.searchsorted(E4M3_MAG, q), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = q - E4M3_MAG[lo], E4M3_MAG[hi] - q
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def mx8_scale(m, ceil):
    """Scale bytes of blocks with the (finite) largest magnitudes m."""
    e = np.frexp(m)[1].astype(np.int64) - 1 - 8
    if ceil:
        e = e + (m > 448 * np.ldexp(1.0, e))
    return np.where(m == 0, 0, np.clip(e, -127, 127) + 127)


def quant_mxfp8(x, ceil):
    """x [R, K] fp64 -> code bytes [R, K], scale bytes [R, K / 32], values [R, K] fp64."""
    R, K = x.shape
    b = np.asarray(x, np.float64).reshape(-1, 32)
    good = np.all(np.isfinite(b), axis=1)
    z = np.where(good[:, None], b, 0.0)
    sf = mx8_scale(np.max(np.abs(z), axis=1), ceil)
    c = e4m3_codes(np.ldexp(z, (127 - sf)[:, None]))
    vals = np.ldexp(np.copysign(E4M3_MAG[c], b), (sf - 127)[:, None])
    codes = np.where(good[:, None], c + 128 * np.signbit(b), 0)
    vals[~good] = np.nan
    return codes.reshape(R, K), np.where(good, sf, 255).reshape(R, K // 32), vals.reshape(R, K)


def decode8(codes, sf):
    """Code bytes [R, K], scale bytes [R, K / 32] -> fp64."""
    c = np.asarray(codes).astype(np.int64)
    v = np.where((c & 127) == 127, np.nan, np.append(E4M3_MAG, 0.0)[c & 127])
    v = np.where(c >= 128, -v, v)
    s = np.asarray(sf).astype(np.int64)
    return v * np.repeat(np.where(s == 255, np.nan, 2.0 ** (np.minimum(s, 254) - 127.0)), 32, axis=1)


def untile(tiled, R, S):
    """Tiled scale bytes -> [R, S]."""
    KA = (S + 3) // 4
    r, b = np.arange(R)[:, None], np.arange(S)[None, :]
    return np.asarray(tiled).reshape(-1)[((r >> 7) * KA + (b >> 2)) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]


def mx8_close(codes, sf, ref, slack, ceil=True):
    """Whether code bytes [R, K] with scale bytes [R, K / 32] are the MXFP8 form of values within `slack`
    (relative, a block's values to their largest) of ref: the scale is that of the largest magnitude, or
    of one within slack of it; an element is within half a step (2^-4 of it, or half of the smallest
    step, 2^-10 scales)."""
    R, K = ref.shape
    m = np.abs(ref).reshape(R, K // 32, 32).max(-1)
    lo, hi = mx8_scale(m * (1 - slack), ceil), mx8_scale(m * (1 + slack), ceil)
    s = np.asarray(sf).astype(np.int64)
    if not np.all((s >= lo) & (s <= hi)):
        return False
    step = np.repeat(2.0 ** (s - 127.0), 32, axis=1)
    off = np.repeat(m * slack, 32, axis=1)
    mag = np.abs(ref) + off
    bound = 2.0 ** -4 * mag + 2.0 ** -10 * step + off
    if not ceil:  # magnitudes past 448 saturate
        bound = np.maximum(bound, mag - 448 * step + off)
    return bool(np.all(np.abs(decode8(codes, s) - ref) <= bound))


# ------------------------------------------------------------------------------- routing

def scores(l, kind):
    """Scores of a token's logits (fp64, NaN counts as -inf)."""
    l = np.where(np.isnan(l), -np.inf, l)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-l))
    m = np.max(l)
    e = np.exp(l - (m if np.isfinite(m) else 0.0))
    return e / e.sum() if e.sum() > 0 else e


def route(logits, bias, k, kind, groups, topg, top2, renorm, scale):
    """logits [T, E] fp64, bias [E] or None -> ids [T, k], weights [T, k] fp64."""
    T, E = logits.shape
    ids, ws = np.zeros((T, k), np.int64), np.zeros((T, k))
    n = E // groups
    for t in range(T):
        l = np.where(np.isnan(logits[t]), -np.inf, logits[t])
        bad = np.isnan(logits[t]).any() or (kind == "softmax" and np.isposinf(l).any())
        if kind == "softmax" and np.isposinf(l).any():
            s = np.isposinf(l) / np.isposinf(l).sum()
        else:
            s = scores(l, kind)
        own = l if bias is None else np.where(np.isneginf(l) | np.isnan(bias), -np.inf, s + np.nan_to_num(bias, nan=0.0, posinf=np.inf, neginf=-np.inf))
        # (the order of scores is that of the logits; sums are of scores)
        part = own if bias is not None or not top2 else np.where(np.isneginf(l), -np.inf, s)
        keep = np.ones(E, bool)
        if groups > 1:
            gs = []
            for g in range(groups):
                v = np.sort(part[g * n:(g + 1) * n])[::-1]
                gs.append(v[0] + v[1] if top2 and n > 1 and v[1] > -np.inf else v[0])
            order = sorted(range(groups), key=lambda g: (-gs[g], g))[:topg]
            keep = np.isin(np.arange(E) // n, order)
        order = sorted(np.flatnonzero(keep), key=lambda e: (-own[e], e))[:k]
        ids[t] = order
        w = s[order]
        if renorm:
            with np.errstate(over="ignore", invalid="ignore", under="ignore"):
                lw = l[order]
                top = np.max(lw)
                if top == -np.inf:
                    w = np.zeros(k)
                else:
                    if kind == "softmax":
                        w = np.exp(lw - top)
                    else:  # relative to the largest: log s = -log(1 + e^-l)
                        ls = -np.logaddexp(0, -lw)
                        w = np.exp(ls - ls.max())
                    w = w / w.sum()
        ws[t] = np.nan if bad else w * scale
    return ids, ws


def route_grad(logits, ids, dw, kind, renorm, scale):
    """dlogits [T, E] fp64 of finite (or -inf) logits: the Jacobian's transpose, position by position."""
    T, E = logits.shape
    k = ids.shape[1]
    out = np.zeros((T, E))
    for t in range(T):
        l = logits[t]
        live = (ids[t] >= 0) & (ids[t] < E)
        pos = ids[t][live].astype(np.int64)
        g = dw[t][live] * scale
        s = scores(l, kind)
        if renorm:
            if not len(pos) or np.all(np.isneginf(l[pos])):
                continue
            ls = l[pos] - l[pos].max() if kind == "softmax" else -np.logaddexp(0, -l[pos])
            q = np.exp(ls - ls.max())
            q /= q.sum()
            f = 1.0 if kind == "softmax" else 1 - s[pos]
            np.add.at(out[t], pos, q * (g - (g * q).sum()) * f)
        elif kind == "sigmoid":
            np.add.at(out[t], pos, g * s[pos] * (1 - s[pos]))
        else:
            d = np.zeros(E)
            np.add.at(d, pos, g)
            out[t] = s * (d - (d * s).sum())
    return out


# ------------------------------------------------------------------------------- norm, gate

def rmsnorm(h, w, eps):
    rstd = 1 / np.sqrt((h ** 2).mean(1) + eps)
    return h * rstd[:, None] * w, rstd


def rmsnorm_grad(dy, h, w, rstd, dh):
    x = h * rstd[:, None]
    d = dy * w
    return rstd[:, None] * (d - x * (d * x).mean(1, keepdims=True)) + dh, (dy * x).sum(0)


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-g))


def swiglu(g, u):
    return g * sigmoid(g) * u


def swiglu_grad(ds, g, u):
    s = sigmoid(g)
    return ds * u * s * (1 + g * (1 - s)), ds * g * s
