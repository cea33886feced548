"""Routing, its gradient, the checkpointed SwiGLU and the combine from their
definitions in binary64 numpy, with the error each f32 evaluation may make.

Shares no code with the kernels.  EPS is half a unit in the last place of f32
relative to the value.
"""
import numpy as np

EPS = 2.0 ** -24


def softmax(x, mask=None):
    """f64 rows [T, E]; (p, routed): p is 0 for tokens that are not routed."""
    x = np.array(x, np.float64)
    if mask is not None:
        x[~np.asarray(mask, bool)] = -np.inf
    bad = np.isnan(x).any(1) | (x == np.inf).any(1)
    x[bad] = -np.inf
    m = x.max(1, keepdims=True)
    routed = m[:, 0] > -np.inf
    e = np.exp(x - np.where(routed[:, None], m, 0.0))
    return e / np.maximum(e.sum(1, keepdims=True), 1e-300), routed, bad


def route(logits, k, norm=True, shared=0, mask=None):
    """The forward definition.  NaN/+inf rows that are not masked: weights of the k choices are NaN."""
    x = np.array(logits, np.float64)
    T, E = x.shape
    kk, G = k + shared, E + shared
    p, routed, bad = softmax(x, mask)
    live = np.where(routed[:, None], x, -np.inf)
    order = np.argsort(-live, axis=1, kind="stable")[:, :k]
    have = np.take_along_axis(live, order, 1) > -np.inf
    w = np.where(have, np.take_along_axis(p, order, 1), 0.0)
    if norm:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    w[bad] = np.nan
    experts = np.where(have, order, -1)
    ids = np.where(routed[:, None], np.arange(E, G)[None, :], -1)
    experts = np.concatenate([experts, ids], 1).astype(np.int32)
    w = np.concatenate([w, np.repeat(routed[:, None].astype(np.float64), shared, 1)], 1)
    flat = experts.reshape(-1)
    counts = np.bincount(flat[flat >= 0], minlength=G)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    perm = np.argsort(np.where(flat >= 0, flat, G), kind="stable")
    R, used = T * kk, int(off[-1])
    src = np.full(R, -1, np.int32)
    src[:used] = perm[:used] // kk
    pos = np.full(R, -1, np.int32)
    pos[perm[:used]] = np.arange(used)
    rw = np.zeros(R)
    rw[:used] = w.reshape(-1)[perm[:used]]
    n = int(routed.sum())
    q = p[routed].sum(0) if not bad.any() else np.full(E, np.nan)
    loss = float(E / (k * n * n) * (counts[:E] * q).sum()) if n else (np.nan if bad.any() else 0.0)
    return dict(experts=experts, weights=w, counts=np.append(counts, n).astype(np.int32), group_offsets=off, src=src,
                pos=pos.reshape(T, kk), row_weights=rw, prob_sum=q, loss=loss)


def logit_span(logits, mask=None):
    """Largest distance of a finite logit from its row's maximum (the exponential's argument)."""
    x = np.array(logits, np.float64)
    if mask is not None:
        x = x[np.asarray(mask, bool)]
    if not x.size:
        return 0.0
    x[~np.isfinite(x)] = np.nan
    ok = ~np.isnan(x).all(1)
    if not ok.any():
        return 0.0
    return float(min(np.nanmax(np.nanmax(x[ok], 1, keepdims=True) - x[ok]), 110.0))   # exp(-110) is 0 in f32


def weight_tol(span, E):
    """Relative error of a softmax weight: the exponential's argument is rounded twice (2 span EPS), the hardware
    exponential is good to two units (4 EPS), the sums to their length in a lane plus the tree (E / 16 + 8) EPS,
    the reciprocal and product to 4 EPS; once for the numerator and once for the sum."""
    return 2 * (2 * span + 16 + E / 16) * EPS


def route_backward(logits, k, fwd, d_rows, d_loss, norm=True, shared=0, mask=None, counts=None):
    """(gradient, sum of the absolute values of its terms): the formula."""
    T, E = np.shape(logits)
    p, routed, _ = softmax(logits, mask)
    p = np.where(routed[:, None], p, 0.0)
    grad, size = np.zeros((T, E)), np.zeros((T, E))
    counts = fwd["counts"] if counts is None else counts
    if d_loss is not None:
        n = max(int(counts[-1]), 1)
        c = counts[:E].astype(np.float64)
        coef = d_loss * E / (k * float(n) * n)
        dot = (p * c).sum(1, keepdims=True)
        grad += coef * p * (c - dot)
        size += abs(coef) * p * (c + dot)
    if d_rows is not None:
        ex, pos = fwd["experts"][:, :k], fwd["pos"][:, :k]
        have = ex >= 0
        at = np.where(have, ex, 0)
        dw = np.where(have, np.asarray(d_rows, np.float64)[np.where(have, pos, 0)], 0.0)
        ps = np.where(have, np.take_along_axis(p, at, 1), 0.0)
        if norm:
            w = ps / np.maximum(ps.sum(1, keepdims=True), 1e-300)
            g = w * (dw - (w * dw).sum(1, keepdims=True))
            s = w * (np.abs(dw) + (w * np.abs(dw)).sum(1, keepdims=True))
        else:
            g, s = ps * dw, ps * np.abs(dw)
            grad -= p * g.sum(1, keepdims=True)
            size += p * s.sum(1, keepdims=True)
        rows = np.repeat(np.arange(T)[:, None], k, 1)
        np.add.at(grad, (rows[have], at[have]), g[have])
        np.add.at(size, (rows[have], at[have]), s[have])
    return grad, size


def objective(logits, k, fwd, d_rows, d_loss, norm=True, mask=None):
    """The scalar whose gradient route_backward is, with fwd's choice and counts held fixed."""
    T, E = np.shape(logits)
    p, routed, _ = softmax(logits, mask)
    p = np.where(routed[:, None], p, 0.0)
    total = 0.0
    if d_loss is not None:
        n = max(int(fwd["counts"][-1]), 1)
        total += d_loss * E / (k * float(n) * n) * (fwd["counts"][:E] * p.sum(0)).sum()
    if d_rows is not None:
        ex, pos = fwd["experts"][:, :k], fwd["pos"][:, :k]
        have = ex >= 0
        w = np.where(have, np.take_along_axis(p, np.where(have, ex, 0), 1), 0.0)
        if norm:
            w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
        total += (w * np.where(have, np.asarray(d_rows, np.float64)[np.where(have, pos, 0)], 0.0)).sum()
    return total


def sigmoid(z):
    return 1.0 / (1.0 + np.exp(-np.asarray(z, np.float64)))


def swiglu(g, u, w):
    return w[:, None] * (g * sigmoid(g) * u)


def swiglu_backward(dh, g, u, w):
    """(dg, du, h, dw) and the size of the terms that dg adds."""
    s = sigmoid(g)
    a, da = g * s, w[:, None] * dh
    dg = da * u * (s + a * (1 - s))
    return dg, da * a, w[:, None] * a * u, (dh * a * u).sum(1), np.abs(da * u) * (s + np.abs(a) * (1 - s))


def bf16(x):
    """f64/f32 -> bf16 bits, nearest even."""
    b = np.asarray(x, np.float32).view(np.uint32)
    return ((b.astype(np.uint64) + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def from_bf16(b):
    return (np.asarray(b, np.uint16).astype(np.uint32) << 16).view(np.float32)


def e4m3_values():
    """The 256 E4M3 values (NaN codes as NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


def mxfp8(x):
    """Rowwise MXFP8 of f64 values [R, K]: smallest k in [-127, 119] with the block within 448 * 2^k, codes to the
    nearest value (ties to the even code), saturating."""
    b = np.asarray(x, np.float64).reshape(len(x), -1, 32)
    top = np.abs(b).max(2)
    m, e = np.frexp(top)
    k = np.clip(np.where(top > 0, e - 9 + (m > 0.875), -127), -127, 119)
    y = np.ldexp(b, -k[:, :, None])
    mag = np.minimum(np.abs(y), 448.0)
    _, ey = np.frexp(mag)
    step = np.ldexp(1.0, np.maximum(ey, -5) - 4)
    q = np.rint(mag / step) * step                  # rint: ties to even
    table = e4m3_values()[:127]
    codes = np.searchsorted(table, q).astype(np.uint8)
    assert np.array_equal(table[codes], q)
    codes |= (np.signbit(y).astype(np.uint8) << 7)
    return codes.reshape(np.shape(x)), (k + 127).astype(np.uint8)


def mxfp8_value(codes, scales):
    v = e4m3_values()[codes].reshape(len(codes), -1, 32)
    return np.ldexp(v, scales.astype(np.int64)[:, :, None] - 127).reshape(codes.shape)


def combine(y, pos, weights=None):
    """(sum, sum of absolute values)."""
    y = np.asarray(y, np.float64)
    ok = (pos >= 0) & (pos < len(y))
    w = np.where(ok, 1.0 if weights is None else np.asarray(weights, np.float64), 0.0)
    rows = y[np.where(ok, pos, 0)]
    return np.einsum("tj,tjh->th", w, rows), np.einsum("tj,tjh->th", np.abs(w), np.abs(rows))
