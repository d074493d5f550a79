"""The layer operators in 64 bits on the CPU, token by token from their
formulas, each with a bound of what 32-bit arithmetic may add (test
infrastructure).

Every function returns (value, bound) pairs: |computed - value| must not pass
the bound plus the final rounding, half a step of the output's type.  U = 2^-24
is half a step of fp32; a bound is a count of roundings times the sum of the
magnitudes they act on, so it holds for any order of the sums.
"""
import numpy as np

U = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def _silu(y, err):
    """silu(y) and its bound: the slope of silu is below 1.1; its evaluation rounds the exponent's argument (2 |y| U
    of the exponential), the exponential, the sum, the reciprocal (hardware ones: 2 U each) and the product."""
    v = y * sigmoid(y)
    return v, 1.1 * err + (2 * np.abs(y) + 8) * U * np.abs(v)


def conv(x, weight, bias, state, silu):
    """x [L, D], weight [D, W], state [W - 1, D]; ((y, bound), final state)."""
    L, D = x.shape
    W = weight.shape[1]
    seen = np.concatenate([state, x])
    y, mag = np.zeros((L, D)), np.zeros((L, D))
    for j in range(W):
        y += weight[:, j] * seen[j: j + L]
        mag += np.abs(weight[:, j] * seen[j: j + L])
    if bias is not None:
        y, mag = y + bias, mag + np.abs(bias)
    err = (W + 1) * U * mag
    if silu:
        y, err = _silu(y, err)
    return (y, err), seen[L:]


def ssm(x, dt, A, Bm, Cm, skip, z, dt_bias, softplus, state):
    """x, dt, z [L, D], A [D, N], Bm, Cm [L, G, N], state [D, N]; ((y, bound), (h, bound)).

    Roundings per token: the step size (argument, exponential, reciprocal, a nine-term series, products: below
    (3 |v| + 24) U relative), the decay's exponent (its product twice rounded: 4 U times its size) and exponential
    (2 U, and as much for each product of decays), the input's two products and the update."""
    L, D = x.shape
    N, G = A.shape[1], Bm.shape[1]
    h, hm, he = state.copy(), np.abs(state), np.zeros((D, N))
    ys, es = np.zeros((L, D)), np.zeros((L, D))
    for t in range(L):
        v = dt[t] + (0 if dt_bias is None else dt_bias)
        step = np.logaddexp(v, 0) if softplus else v
        dstep = ((3 * np.abs(v) + 24) if softplus else 1 + 0 * v) * U
        B, C = np.repeat(Bm[t], D // G, 0), np.repeat(Cm[t], D // G, 0)
        a = np.exp(step[:, None] * A)
        b = (step * x[t])[:, None] * B
        da = np.abs(step[:, None] * A) * (dstep[:, None] + 6 * U) + 8 * U
        db = dstep[:, None] + 6 * U
        he = a * he + a * hm * da + np.abs(b) * db
        h, hm = a * h + b, a * hm + np.abs(b)
        y, e = (h * C).sum(1), (he * np.abs(C)).sum(1) + (N + 2) * U * (hm * np.abs(C)).sum(1)
        if skip is not None:
            y, e = y + skip * x[t], e + 2 * U * (np.abs(y) + np.abs(skip * x[t]))
        if z is not None:
            s, ds = _silu(z[t], 0 * z[t])
            y, e = y * s, e * np.abs(s) + np.abs(y) * ds + 2 * U * np.abs(y * s)
        ys[t], es[t] = y, e
    return (ys, es), (h, he)


def rotary(x, theta, interleaved, scale, inverse):
    """x [..., T, H, d], theta [..., T, pairs]; (y, bound): cosine and sine are within 4 U, the two products and
    their sum round three times."""
    pairs = theta.shape[-1]
    y, err = x.copy(), np.zeros_like(x)
    c, s = scale * np.cos(theta)[..., None, :], scale * np.sin(theta)[..., None, :] * (-1 if inverse else 1)
    iu = np.arange(pairs) * 2 if interleaved else np.arange(pairs)
    iv = iu + (1 if interleaved else pairs)
    u, v = x[..., iu], x[..., iv]
    y[..., iu], y[..., iv] = u * c - v * s, v * c + u * s
    err[..., iu] = err[..., iv] = 8 * U * abs(scale) * (np.abs(u) + np.abs(v))
    return y, err


def delta_step(q, k, v, log_alpha, beta, S, erase=True, exclusive=False, gate=None, weight=None, eps=0.0):
    """q, k [H, dk], v [H, dv], S [H, dv, dk]; ((o, bound), (S', bound)).  Roundings: a unit vector 8 U, a dot over dk
    9 more, the decay 3, the write strength 4 more: below 32 U of the state's magnitudes, 48 U of the readout's."""
    q = q / np.maximum(np.linalg.norm(q, axis=-1, keepdims=True), 1e-6)
    k = k / np.maximum(np.linalg.norm(k, axis=-1, keepdims=True), 1e-6)
    a = np.exp(log_alpha)[:, None, None]
    b = beta[:, None]
    ks, ksm = a[..., 0] * np.einsum("hij,hj->hi", S, k), a[..., 0] * np.einsum("hij,hj->hi", np.abs(S), np.abs(k))
    w, wm = (b * (v - ks), np.abs(b) * (np.abs(v) + ksm)) if erase else (b * v, np.abs(b * v))
    new, newm = a * S + w[..., None] * k[:, None], a * np.abs(S) + wm[..., None] * np.abs(k)[:, None]
    read, readm = (a * S, a * np.abs(S)) if exclusive else (new, newm)
    o, om = np.einsum("hij,hj->hi", read, q), np.einsum("hij,hj->hi", readm, np.abs(q))
    oe = 48 * U * om
    if gate is not None:
        ms = (o * o).mean(-1, keepdims=True) + eps
        inv = 1 / np.sqrt(ms)
        rel = (np.abs(o) * oe).mean(-1, keepdims=True) / ms + 16 * U
        g = weight * sigmoid(gate) * inv
        oe = np.abs(g) * (oe + np.abs(o) * (rel + (2 * np.abs(gate) + 16) * U))
        o = g * o
    return (o, oe), (new, 32 * U * newm)


def check(got, want, bound, kind, what=""):
    """got (any float array) against want within bound plus half a step of `kind` ("bf16" or "f32")."""
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{what}: non-finite values"
    tol = bound * (1 + HALF_STEP[kind]) + HALF_STEP[kind] * np.abs(want) + 1e-37
    off = np.abs(got - want) - tol
    if off.size and off.max() > 0:
        i = np.unravel_index(off.argmax(), off.shape)
        raise AssertionError(f"{what}: at {i} got {got[i]!r}, want {want[i]!r} +- {tol[i]:.3e}")
