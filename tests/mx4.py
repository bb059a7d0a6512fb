"""Plain forms of the MX4 operators for the tests: numpy, 64 bits (the rotation in
fp32 with the defined order of butterflies, since the order is part of the
definition).  Shared by the CPU and GPU tests; nothing here uses the library."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def rotate(x, g, sign_in=None, sign_out=None):
    """fp32 rows (M, K) . diag(sign_in) H_g diag(sign_out) / sqrt(g), butterflies of
    distance 1, 2, 4, ... in fp32, one fp32 multiplication at the end."""
    v = np.ascontiguousarray(x, np.float32).reshape(-1, g)
    if sign_in is not None:
        v = v * np.where(np.asarray(sign_in) < 0, np.float32(-1), np.float32(1))
    d = 1
    while d < g:
        v = v.reshape(-1, g // (2 * d), 2, d)
        v = np.stack([v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]], 2)
        d *= 2
    v = v.reshape(-1, g) * np.float32(1.0 / np.sqrt(np.float64(g)))
    if sign_out is not None:
        v = v * np.where(np.asarray(sign_out) < 0, np.float32(-1), np.float32(1))
    return v.reshape(x.shape)


def scale_exponent(amax):
    """X of blocks with largest magnitude amax (finite, 64 bits): floor(log2) - 2, at least -127."""
    m, e = np.frexp(np.asarray(amax, np.float64))
    return np.where(np.asarray(amax) > 0, np.maximum(e - 1 - 2, -127), -127)


def nearest_code(v):
    """Magnitude codes of |v| (64 bits, already divided by the scale): nearest, ties to even, saturated."""
    v = np.abs(v)
    hi = np.minimum(np.searchsorted(GRID, v), 7)
    lo = np.maximum(hi - 1, 0)
    dh, dl = GRID[hi] - v, v - GRID[lo]
    return np.where(v >= 6, 7, np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo))


def quantize(y):
    """(M, K) values -> (codes (M, K/2), scale bytes in rows (M, K/32))."""
    M, K = y.shape
    b = np.asarray(y, np.float64).reshape(M, K // 32, 32)
    with np.errstate(invalid="ignore"):
        amax = np.abs(b).max(-1)
        bad = ~np.isfinite(amax)
        X = scale_exponent(np.where(bad, 1.0, amax))
        c = nearest_code(np.where(bad[..., None], 0, b) * np.exp2(-X.astype(np.float64))[..., None])
    c = np.where(bad[..., None], 0, c | (np.signbit(b) << 3)).astype(np.uint8).reshape(M, K)
    return c[:, 0::2] | (c[:, 1::2] << 4), np.where(bad, 255, X + 127).astype(np.uint8)


def slabs(rows):
    """Scale bytes in rows (..., rows, K/32) -> slabs (..., ceil(K/256), rows, 8)."""
    *lead, R, B = rows.shape
    S = -(-B // 8)
    p = np.zeros((*lead, R, 8 * S), np.uint8)
    p[..., :B] = rows
    return np.ascontiguousarray(np.moveaxis(p.reshape(*lead, R, S, 8), -2, -3))


def unslab(s, K):
    *lead, S, R, _ = s.shape
    return np.moveaxis(s, -3, -2).reshape(*lead, R, 8 * S)[..., :K // 32]


def values(codes, scale_rows):
    """The 64-bit values of codes (..., rows, K/2) with scale bytes in rows."""
    K = codes.shape[-1] * 2
    n = np.empty((*codes.shape[:-1], K), np.int64)
    n[..., 0::2], n[..., 1::2] = codes & 15, codes >> 4
    v = GRID[n & 7] * np.where(n & 8, -1.0, 1.0)
    s = np.where(scale_rows == 255, np.nan, np.exp2(scale_rows.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def product_bound(a, w):
    """Bound on the fp32 error of a @ w.T: one rounding per 32 k, and a few more,
    of partial sums no larger than sum |a w|."""
    return (a.shape[1] / 32 + 8) * 2.0 ** -24 * (np.abs(a) @ np.abs(w).T)


# half a unit in the last place, relative, and the smallest absolute step of a type
HALF_ULP = {"f32": (2.0 ** -24, 2.0 ** -149), "f16": (2.0 ** -11, 2.0 ** -24), "bf16": (2.0 ** -8, 2.0 ** -133)}


def close(got, ref, bound, dtype):
    """Every finite reference within bound plus the rounding to dtype (twice half a
    unit: the rounding of a value that is itself off), NaN where the reference is."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    rel, step = HALF_ULP[dtype]
    err = np.abs(got[ok] - ref[ok])
    lim = (np.broadcast_to(bound, ref.shape)[ok]) * (1 + 2 * rel) + rel * np.abs(ref[ok]) + step
    assert (err <= lim).all(), f"{int((err > lim).sum())} of {err.size} beyond the bound, worst {np.max(err / lim):.3g}"


def route(logits, k, renormalize=True):
    """(weights, experts, rows, pos, offsets) one token at a time, 64 bits."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    experts, weights = np.full((T, k), -1, np.int64), np.zeros((T, k))
    for t in range(T):
        live = [e for e in range(E) if l[t, e] > -np.inf]
        top = sorted(live, key=lambda e: (-l[t, e], e))[:k]
        if not top:
            continue
        p = np.exp(l[t, top] - l[t, top[0]])
        total = p.sum() if renormalize else np.exp(l[t, live] - l[t, top[0]]).sum()
        experts[t, :len(top)] = top
        weights[t, :len(top)] = p / total
    flat = experts.reshape(-1)
    order = [s for e in range(E) for s in np.nonzero(flat == e)[0]]
    rows, pos = np.full(T * k, -1, np.int64), np.full(T * k, -1, np.int64)
    rows[:len(order)] = np.array(order, np.int64) // k
    pos[order] = np.arange(len(order))
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    return weights, experts, rows, pos.reshape(T, k), offsets


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))
