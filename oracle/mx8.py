"""Plain float64 (numpy) definitions of the MXFP8 operators: block conversion, RMS norm and the
expert FFN with MXFP8 activations, each with the interval that fp32 arithmetic may reach.

A result that is rounded to E4M3 moves by a whole step when fp32 arithmetic and this one fall on
two sides of a rounding boundary, so the checks here carry an interval: `span(v, err)` gives the
least and greatest MXFP8 value that any number within err of v can be rounded to.
"""
import numpy as np

# the 127 non-negative E4M3 values, by code
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def scale_stride(d):
    return (d + 127) // 128 * 4


def _scale_of(amax):
    """Scale bytes of blocks with the largest magnitudes amax (255 where not finite)."""
    amax = np.asarray(amax, dtype=np.float64)
    ok = np.isfinite(amax)
    e = np.frexp(np.where(ok & (amax > 0), amax, 1.0))[1] - 1  # floor(log2)
    s = np.where(amax > 0, np.maximum(e - 8 + 127, 0), 0)
    return np.where(ok, s, 255).astype(np.uint8)


def _codes(v, s):
    """E4M3 codes of v / 2^(s - 127), nearest, ties to even, saturating; v [..., 32], s [...]."""
    q = v / np.exp2(s.astype(np.float64) - 127.0)[..., None]
    a = np.minimum(np.abs(q), 448.0)
    hi = np.clip(np.searchsorted(E4M3, a, side="left"), 1, 126)
    up, down = E4M3[hi] - a, a - E4M3[hi - 1]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
    return (c | np.where(np.signbit(q), 128, 0)).astype(np.uint8)


def quantize(x):
    """(codes [rows, d], scales [rows, d/32]) of x [rows, d]."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    with np.errstate(invalid="ignore"):
        amax = np.where(np.isfinite(b).all(-1), np.abs(b).max(-1, initial=0.0), np.inf)
    s = _scale_of(amax)
    bad = s == 255
    c = _codes(np.where(bad[..., None], 0.0, b), np.where(bad, 127, s))
    c[bad] = 0x7F
    return c.reshape(x.shape), s


def dequantize(codes, scales):
    m = codes & 0x7F
    v = np.where(m == 0x7F, np.nan, E4M3[np.minimum(m, 126)]) * np.where(codes & 0x80, -1.0, 1.0)
    x = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    return (v.reshape(codes.shape[0], -1, 32) * x[..., None]).reshape(codes.shape)


def pack(codes, scales):
    """The byte buffer of rows: codes, then scales with every row filled up to whole words."""
    rows, d = codes.shape
    s = np.zeros((rows, scale_stride(d)), dtype=np.uint8)
    s[:, :d // 32] = scales
    return np.concatenate([codes.reshape(-1), s.reshape(-1)])


def unpack(buf, rows, d):
    buf = np.asarray(buf, dtype=np.uint8)
    return (buf[:rows * d].reshape(rows, d),
            buf[rows * d:rows * (d + scale_stride(d))].reshape(rows, -1)[:, :d // 32])


def span(v, err):
    """(least, greatest) value in MXFP8 of numbers within err of v, both [rows, d] (finite): the
    block's scale may be any that its largest magnitude may have, each element any value
    between the conversions of v - err and v + err under these scales."""
    rows, d = v.shape
    b, e = v.reshape(rows, -1, 32), np.broadcast_to(err, v.shape).reshape(rows, -1, 32)
    top = np.abs(b)
    lo, hi = None, None
    for s in (_scale_of(np.maximum(top - e, 0).max(-1)), _scale_of((top + e).max(-1))):
        for w in (b - e, b + e):
            q = dequantize(_codes(w, s).reshape(rows, d), s)
            lo = q if lo is None else np.minimum(lo, q)
            hi = q if hi is None else np.maximum(hi, q)
    return lo, hi


def rmsnorm(s, gamma, eps):
    """(y, bound of the fp32 error) of rows s [T, d] in float64.  The squares' sum has one rounding
    a product and addition of positive terms: at most 8 d / 8192 + 32 in a thread, then under 32
    over threads and waves; the mean, root, quotient and two products add under 8."""
    s, gamma = np.asarray(s, dtype=np.float64), np.asarray(gamma, dtype=np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        y = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * gamma
    return y, (72 + s.shape[-1] / 1024) * 2.0 ** -24 * np.abs(y)


# A matrix instruction adds groups of 16 products to an fp32 accumulator.  One fp32 step (2^-23)
# of the sum of the magnitudes is taken for each instruction, a few more for sums over waves.
# Inside a group it aligns the products to the largest and drops what lies 13 binary places
# below it (measured: 256 + 2^-5 is exact, 256 + 2^-6 is 256).  A product has 6 significant bits,
# so only those under 2^-6 of the largest lose any, and at most 2^-12 of it.
def _sum_err(x, w):
    """Bound of |fp32 x w^T - exact| for x [n, K], w [R, K]."""
    x, w = np.abs(x), np.abs(w)
    K = x.shape[1]
    err = (K / 64 + 8) * 2.0 ** -23 * (x @ w.T)
    for r in range(len(x)):
        p = (x[r] * w).reshape(len(w), -1, 16)
        top = p.max(-1, keepdims=True)
        err[r] += np.where(p < 2.0 ** -6 * top, np.minimum(p, 2.0 ** -12 * top), 0).sum((1, 2))
    return err


def expert_ffn(x, perm, k, offsets, weights):
    """(y, tolerance before its rounding) of the grouped rows [T*k, d]: x [T, d] the values of the
    MXFP8 rows, weights: {expert: (gate [f, d], up [f, d], down [d, f])} in float64."""
    A, d = len(perm), x.shape[1]
    y, tol = np.zeros((A, d)), np.zeros((A, d))
    for e, (wg, wu, wd) in weights.items():
        r0, r1 = int(offsets[e]), int(offsets[e + 1])
        if r0 == r1:
            continue
        X = x[perm[r0:r1] // k]
        nan = np.isnan(X).any(1)
        X = np.where(nan[:, None], 0.0, X)
        g, u = X @ wg.T, X @ wu.T
        dg, du = _sum_err(X, wg), _sum_err(X, wu)
        with np.errstate(over="ignore"):
            silu = g / (1.0 + np.exp(-g))
        h = silu * u
        # |silu'| <= 1.1; the exponential, reciprocal and products: (16 + |g|) steps of 2^-23
        dh = (1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + (16 + np.abs(g)) * 2.0 ** -23 * np.abs(h))
        q = dequantize(*quantize(h))
        lo, hi = span(h, dh)
        off = np.maximum(hi - q, q - lo)
        y[r0:r1] = q @ wd.T
        tol[r0:r1] = off @ np.abs(wd).T + _sum_err(np.abs(q) + off, wd)
        y[r0:r1][nan] = np.nan
    return y, tol
