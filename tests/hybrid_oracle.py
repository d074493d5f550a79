"""The paged cache, a new token's attention over it and the seam between two
blocks in 64 bits on the CPU, from their formulas, with a bound of what 32-bit
arithmetic may add (test infrastructure; conventions of layer_oracle.py).
"""
import numpy as np

from layer_oracle import U

# ---- formats: 32 channels share a power of two, each channel is a code ----

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127])
TABLE = {"mxfp8": E4M3, "mxfp4": E2M1}


def encode(x, form):
    """x [..., d] -> (codes [..., d] with the sign as their top bit, scale bytes [..., d / 32])."""
    table = TABLE[form]
    b = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(np.isfinite(b), b, 0.0)
    top = np.abs(b).max(-1)
    e = np.full(top.shape, -110)
    while (top > table[-1] * 2.0 ** e).any():  # the least that fits
        e = e + (top > table[-1] * 2.0 ** e)
    a = np.abs(b) / (2.0 ** e)[..., None]
    hi = np.searchsorted(table, a).clip(0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - a, a - table[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(table[hi] == a, hi, code) + (np.signbit(b) * (128 if form == "mxfp8" else 8))
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def decode(codes, scales, form):
    table, sign = TABLE[form], 128 if form == "mxfp8" else 8
    v = np.append(table, np.nan)[codes % sign] * np.where(codes >= sign, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v.reshape(*codes.shape[:-1], -1, 32) * s[..., None]).reshape(codes.shape)


# ---- attention of one token ----

def attend(q, k, v, scale, short):
    """q [G, d], k, v [n, d]; (out, bound) [G, d], (lse, bound) [G].

    A score is a product of d terms and a scale: (d + 4) U of the magnitudes.  A weight e^(s - m) takes that error, the
    rounding of its exponent's argument (2 U |s - m|, twice) and 8 U.  Weights enter products exactly, as fp32 or three
    16-bit terms; ``short`` (rows in 16 bits) allows them 2^-16 all the same, far below an output's last digit.  The sums
    over n tokens round at most n + 64 times.

    Below the least normal number, 2^-126, fp32 gives up digits.  A weight (at most 1, the largest is 1, so z >= 1) that
    lies there is taken for something between zero and 2^-126, so it is off by 2^-126 at most; so are the two factors,
    at most 1, by which waves' and items' parts come to one maximum: 3 * 2^-126 sum |v| in all.  A product with a value
    that lies there may vanish: another 2^-126 a token."""
    G, d = q.shape
    if len(k) == 0:
        return (np.zeros((G, d)), np.zeros((G, d))), (np.full(G, -np.inf), np.zeros(G))
    s, sm = scale * q @ k.T, abs(scale) * np.abs(q) @ np.abs(k).T
    m = s.max(1, keepdims=True)
    w = np.exp(s - m)
    z = w.sum(1, keepdims=True)
    w = w / z
    ds = (d + 4) * U * sm
    rel = ds + (4 * np.abs(s - m) + 8) * U + (2.0 ** -16 if short else 2.0 ** -22)
    n = len(k) + 64
    zerr = (w * rel).sum(1, keepdims=True) + n * U
    out = w @ v
    err = (w * (rel + zerr + n * U)) @ np.abs(v) + 2.0 ** -126 * (3 * np.abs(v).sum(0) + n)
    lse = (m + np.log(z))[:, 0]
    return (out, err), (lse, zerr[:, 0] + ds.max(1) + 4 * U * (np.abs(m[:, 0]) + np.abs(lse) + 1))


def visible(length, reach, window, sinks):
    n = min(max(length, 0), reach)
    p = np.arange(n)
    return p if not window else p[(p >= n - window) | (p < sinks)]


# ---- the seam ----
# K roundings: a row's mean of squares (chains of up to 16 terms, then sums over lanes and waves: 40, half of that
# through the root), root and quotient, and the products around them: below 64 in each of the two norms.  `cond` is what
# cancellation in h = a x + g u amplifies them by.
K = 64


def seam(x, y, gate, post, weight, alpha, eps):
    """Rows x, y [R, D], gate [R, D] or [D]; ((h, bound), (n, bound)); bound of n is None without weight."""
    u = y
    if y is None:
        h, mag = alpha * x, np.abs(alpha * x)
    else:
        if post is not None:
            u = post * y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        g = 1.0 if gate is None else gate
        h, mag = alpha * x + g * u, np.abs(alpha * x) + np.abs(g * u)
    herr = K * U * mag
    if weight is None:
        return (h, herr), None
    ms = (h * h).mean(-1, keepdims=True) + eps
    n = weight * h / np.sqrt(ms)
    rel = np.sqrt((herr * herr).mean(-1, keepdims=True) / ms) + K * U
    return (h, herr), (n, np.abs(weight) * herr / np.sqrt(ms) + np.abs(n) * rel)


def seam_backward(dh, dn, x, y, gate, post, weight, alpha, eps, groups=None):
    """Gradients from the formulas: a dict of (value, bound).  ``groups``: row ranges that have a gate of their own."""
    R, D = x.shape
    out = {}
    g = 1.0 if gate is None else gate
    yh = u = ry = None
    if y is not None:
        ry = 1 / np.sqrt((y * y).mean(-1, keepdims=True) + eps) if post is not None else 1.0
        yh = y * ry
        u = yh * (post if post is not None else 1.0)
    h = alpha * x + (0 if y is None else g * u)
    mag = np.abs(alpha * x) + (0 if y is None else np.abs(g * u))
    dH = np.zeros_like(x) if dh is None else dh.copy()
    err = np.abs(dH) * U
    n_sum = R + K  # roundings of a sum over rows
    if weight is not None:
        ms = (h * h).mean(-1, keepdims=True) + eps
        r = 1 / np.sqrt(ms)
        cond = np.maximum(1.0, np.sqrt((mag * mag).mean(-1, keepdims=True) / ms))
        hh, hm = h * r, mag * r
        a = weight * dn
        c, cm = (a * hh).mean(-1, keepdims=True), (np.abs(a) * hm).mean(-1, keepdims=True)
        dH = dH + r * (a - hh * c)
        err = err + 4 * K * U * cond * (np.abs(dH) + r * (np.abs(a) + hm * cm))
        t, tm = dn * hh, np.abs(dn) * hm * cond
        out["dweight"] = t.sum(0), (n_sum + 2 * K) * U * tm.sum(0)
    out["dx"] = alpha * dH, abs(alpha) * err + U * np.abs(alpha * dH)
    if y is None:
        return out
    if gate is not None:
        t, te = dH * u, err * np.abs(u) + 2 * K * U * np.abs(dH * u)
        te = te + n_sum * U * np.abs(t)
        if groups is None:
            out["dgate"] = t.sum(0), te.sum(0)
        else:
            out["dgate"] = np.stack([t[lo:hi].sum(0) for lo, hi in groups]), np.stack([te[lo:hi].sum(0) for lo, hi in groups])
    du, due = g * dH, np.abs(g) * (err + U * np.abs(dH))
    if post is None:
        out["dy"] = du, due
        return out
    t = du * yh
    out["dpost"] = t.sum(0), ((due + (n_sum + 2 * K) * U * np.abs(du)) * np.abs(yh)).sum(0)
    b, be = post * du, np.abs(post) * (due + U * np.abs(du))
    c, cm = (b * yh).mean(-1, keepdims=True), (np.abs(b * yh)).mean(-1, keepdims=True)
    ce = (be * np.abs(yh)).mean(-1, keepdims=True)
    out["dy"] = ry * (b - yh * c), ry * (be + np.abs(yh) * ce + 2 * K * U * (np.abs(b) + np.abs(yh) * cm))
    return out
