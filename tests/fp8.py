"""Plain forms of the block-scaled fp8 operators and of routing by scores for the
tests: numpy, 64 bits.  Shared by the CPU and GPU tests; nothing here uses the
library."""
import numpy as np

# the magnitudes of codes 0 .. 126 (127 is NaN)
GRID = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])
LEAST = 448 * 2.0 ** -126


def blocks(n):
    return -(-n // 128)


def nearest_code(v):
    """Magnitude codes of |v|: nearest, ties to the even code, at most 126."""
    v = np.abs(v)
    hi = np.minimum(np.searchsorted(GRID, v), 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = np.abs(GRID[hi] - v), v - GRID[lo]
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (v >= 448), hi, lo)


def tops(y, rows):
    """Largest magnitude of every block of `rows` x 128 of y, for each element: (M, K)."""
    M, K = y.shape
    p = np.zeros((-(-M // rows) * rows, blocks(K) * 128))
    p[:M, :K] = np.abs(y)
    b = p.reshape(p.shape[0] // rows, rows, -1, 128).max((1, 3))
    return b, np.repeat(np.repeat(b, rows, 0), 128, 1)[:M, :K]


def quantize(y, rows=1):
    """(M, K) values -> (codes uint8 (M, K), scales float64 (blocks of M, blocks of K));
    rows = 1: activations (their scales are kept transposed), 128: weights."""
    y = np.asarray(y, np.float64)
    with np.errstate(invalid="ignore"):
        bad, every = tops(y, rows)
        A, top = np.maximum(bad, LEAST), np.maximum(every, LEAST)
        fine = np.isfinite(every)
        c = nearest_code(np.where(fine, y, 0) * 448 / np.where(fine, top, 1))
    codes = np.where(fine, c | (np.signbit(y) << 7), 0).astype(np.uint8)
    return codes, np.where(np.isfinite(bad), A / 448, np.nan)


def code_values(codes):
    n = codes.astype(np.int64)
    v = np.append(GRID, np.nan)[n & 127]
    return np.where(n & 128, -v, v)


def values(codes, scales, rows=1):
    """64-bit values; scales (blocks of M, blocks of K)."""
    M, K = codes.shape[-2:]
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), rows, -2)[..., :M, :], 128, -1)[..., :K]
    return code_values(codes) * s


def product_bound(a, w, out="bf16"):
    """Bound on the error of a @ w.T before it is rounded to `out`.  fp32: 128 terms of
    a block in any order, one rounding per block, the scales' product, each of at most
    2^-24 of sum |a w|.  Else the matrix core adds eight neighbouring products in fixed
    point first: each of the eight is off by less than a last place, 2^-13 of the
    largest product, which max |a| max |w| bounds."""
    a, w = np.abs(a), np.abs(w)
    bound = (128 + blocks(a.shape[1]) + 4) * 2.0 ** -24 * (a @ w.T)
    if out == "f32":
        return bound
    tops = lambda v: v.reshape(v.shape[0], v.shape[1] // 8, 8).max(2)  # noqa: E731
    return bound + 8 * 2.0 ** -13 * (tops(a) @ tops(w).T)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def check_gated(codes, scales, g, u, eg, eu):
    """fp8 form (scales (R, blocks)) of silu(g) u, g and u known up to eg and eu: a
    block's scale within the error of its largest value, a code between those of the
    value's bounds."""
    v = silu(g) * u
    # |silu'| <= 1.1; exp's argument, exp, reciprocal and two products: (|g| + 5) 2^-23
    err = 1.1 * np.abs(u) * eg + np.abs(silu(g)) * eu + 1.1 * eg * eu + (np.abs(g) + 5) * 2.0 ** -23 * np.abs(v) + 2.0 ** -126
    R, F = v.shape
    b = lambda t: t.reshape(R, F // 128, 128)  # noqa: E731
    A = np.asarray(scales, np.float64) * 448
    lo, hi = np.maximum(np.abs(v) - err, 0), np.abs(v) + err
    tiny = 2.0 ** -22   # the scale's and the ratio's roundings
    assert (A >= np.maximum(b(lo).max(-1), LEAST) * (1 - tiny)).all() and (A <= np.maximum(b(hi).max(-1), LEAST) * (1 + tiny)).all()
    s = (A / 448)[..., None]
    m = np.abs(b(code_values(codes)))
    least, most = GRID[nearest_code(b(lo) / s * (1 - tiny))], GRID[nearest_code(b(hi) / s * (1 + tiny))]
    assert ((m >= least) & (m <= most)).all()
    sure = (np.abs(v) > err) & (code_values(codes) != 0)
    assert (np.signbit(code_values(codes)) == np.signbit(v))[sure].all()


def route(logits, k, scores="softmax", bias=None, groups=1, top_groups=None, group_best=1, renormalize=True, scale=1.0):
    """(weights, experts, rows, pos, offsets) one token at a time, 64 bits."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    size, top_groups = E // groups, groups if top_groups is None else top_groups
    experts, weights = np.full((T, k), -1, np.int64), np.zeros((T, k))
    for t in range(T):
        live = [e for e in range(E) if l[t, e] > -np.inf]
        s = np.zeros(E)
        if scores == "sigmoid":
            with np.errstate(over="ignore"):
                s[live] = 1 / (1 + np.exp(-l[t, live]))
        elif live:
            top = l[t, live].max()
            with np.errstate(invalid="ignore"):
                s[live] = np.where(l[t, live] == top, 1.0, np.exp(l[t, live] - top))
            s /= s.sum()
        v = s + (0.0 if bias is None else np.asarray(bias, np.float64))
        order = l[t] if bias is None else v
        live = [e for e in live if v[e] > -np.inf]
        if top_groups < groups:
            worth = {}
            for g in range(groups):
                of = l[t] if bias is None and group_best == 1 else v   # the largest is known by its logit
                two = sorted((of[e] for e in live if e // size == g), reverse=True)[:group_best]
                if two:
                    worth[g] = sum(two)
            kept = sorted(worth, key=lambda g: (-worth[g], g))[:top_groups]
            live = [e for e in live if e // size in kept]
        best = sorted(live, key=lambda e: (-order[e], e))[:k]
        w = s[best]
        if renormalize:
            w = w / w.sum() if len(best) and w.sum() > 0 else np.zeros(len(best))
        experts[t, :len(best)], weights[t, :len(best)] = best, w * scale
    flat = experts.reshape(-1)
    order = [i for e in range(E) for i in np.nonzero(flat == e)[0]]
    rows, pos = np.full(T * k, -1, np.int64), np.full(T * k, -1, np.int64)
    rows[:len(order)] = np.array(order, np.int64) // k
    pos[order] = np.arange(len(order))
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    return weights, experts, rows, pos.reshape(T, k), offsets
