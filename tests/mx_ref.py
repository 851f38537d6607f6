"""Plain forms of the microscaled (MX) operators and of the experts' layer, in
64 bits with numpy, from their definitions."""
import numpy as np

E2M1, E4M3 = 1, 2
_MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1_VALUES = np.concatenate([_MAG, -_MAG])


def e4m3_values():
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if (c & 127) == 127 else v
        if c >> 7:
            out[c] = -out[c]
    return out


E4M3_VALUES = e4m3_values()


def pitch(K):
    return (K // 32 + 3) // 4 * 4


def row_bytes(fmt, K):
    return K // 2 if fmt == E2M1 else K


def unpack(codes, fmt):
    """Element values float64 [rows][K] of code bytes."""
    if fmt == E2M1:
        c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
        return E2M1_VALUES[c]
    return E4M3_VALUES[codes]


def values(codes, scales, fmt):
    v = unpack(codes, fmt)
    s = scales[:, :v.shape[1] // 32].astype(np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return v * np.repeat(f, 32, axis=1)


def quantize(x, fmt):
    """(codes, scales) of rows x (float32 values), element by element: every
    grid value's distance, the nearest, ties to the even code."""
    rows, K = x.shape
    b = x.astype(np.float64).reshape(rows, K // 32, 32)
    big = np.max(np.abs(b), -1)
    ok = np.isfinite(b).all(-1)
    big = np.where(ok, big, 1.0)
    # the exponent field of a float32: 0 for zeros and subnormal numbers
    field = np.maximum(np.frexp(big)[1] + 126, 0)
    field = np.where(big < 2.0 ** -126, 0, field)
    s = np.maximum(field - (2 if fmt == E2M1 else 8), 0)
    y = np.where(ok[..., None], b, 0.0) * np.ldexp(1.0, 127 - s)[..., None]
    grid = _MAG if fmt == E2M1 else E4M3_VALUES[:127]
    a = np.minimum(np.abs(y), grid[-1])
    hi = np.clip(np.searchsorted(grid, a), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    neg = np.signbit(b) & ok[..., None]
    code = (code + neg * (8 if fmt == E2M1 else 128)) * ok[..., None]
    code = code.reshape(rows, K).astype(np.uint8)
    if fmt == E2M1:
        code = code[:, 0::2] | (code[:, 1::2] << 4)
    scales = np.zeros((rows, pitch(K)), np.uint8)
    scales[:, :K // 32] = np.where(ok, s, 255)
    return code, scales


def silu_mul(g, u):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def sums_bound(K):
    """Error of a product's float32 sum, of sum |x w|: an instruction adds 64
    inputs or more and drops less than a unit of the 24th bit, e4m3 rows take two
    of them for the same inputs; 4 more for the sums of waves or splits."""
    return (K / 32 + 4) * 2.0 ** -23


def product(x, w, silu):
    """Outputs float64 and the bound on a float32 kernel's error."""
    y, a = x @ w.T, np.abs(x) @ np.abs(w).T
    e = a * sums_bound(x.shape[1])
    if not silu:
        return y, e
    M = w.shape[0] // 2
    g, u, eg, eu = y[:, :M], y[:, M:], e[:, :M], e[:, M:]
    out = silu_mul(g, u)
    # |d silu| <= 1.1; exponential, sum, quotient and two products: 8 roundings
    return out, 1.1 * eg * (np.abs(u) + eu) + np.abs(silu_mul(g, 1.0)) * eu + 8 * 2.0 ** -24 * np.abs(out) + 2.0 ** -126


def route(x, top, renorm):
    """ids, weights (float64) of rows of logits (float64)."""
    rows, E = x.shape
    ids = np.full((rows, top), -1, np.int32)
    w = np.zeros((rows, top))
    for n in range(rows):
        r = x[n]
        if np.isnan(r).any() or (r == np.inf).any():
            w[n] = np.nan
            continue
        order = np.lexsort((np.arange(E), -r))
        best = [e for e in order[:top] if r[e] > -np.inf]
        if not best:
            continue
        m = r[best[0]]
        z = np.exp(r[best] - m).sum() if renorm else np.exp(r - m).sum()
        ids[n, :len(best)] = best
        w[n, :len(best)] = np.exp(r[best] - m) / z
    return ids, w


def plan(ids, experts):
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    at = np.argsort(key, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=experts + 1)[:experts])]).astype(np.int32)
    order = np.where(np.arange(flat.size) < offsets[-1], at, -1).astype(np.int32)
    slots = np.full(flat.size, -1, np.int32)
    slots[at[:offsets[-1]]] = np.arange(offsets[-1])
    return offsets, order, slots.reshape(ids.shape)


def combine(y, slots, weights):
    """Outputs float64 and sum |w y| for the bound."""
    rows, top = slots.shape
    out, mag = np.zeros((rows, y.shape[1])), np.zeros((rows, y.shape[1]))
    for j in range(top):
        s = slots[:, j]
        ok = (s >= 0) & (s < y.shape[0])
        v = np.where(ok[:, None], y[np.where(ok, s, 0)], 0.0)
        out += weights[:, j:j + 1] * v
        mag += np.abs(weights[:, j:j + 1] * v)
    return out, mag
