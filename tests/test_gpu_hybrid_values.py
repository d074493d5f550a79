"""What a new token's attention makes of its weights and of values at the ends of
the number formats, on the GPU: the weights' digits, far and infinite values,
blocks whose scale is NaN or the least there is, queries beyond 16 bits' range,
long sums in fp32."""
import numpy as np
import pytest

import hybrid_oracle as oracle
from layer_oracle import U
from test_gpu_hybrid import i32, n, to_pool
from test_gpu_layer import Rng, _dtype, _torch

pytestmark = pytest.mark.gpu


def cache_of(k, v, form):
    """(cache of k, v [pages, heads, page, d], the values it holds)."""
    torch = _torch()
    if form in ("bf16", "f32"):
        k, v = (torch.from_numpy(a.astype(np.float32)).to(_dtype(form)).cuda() for a in (k, v))
        return (k, v), n(k), n(v)
    enc = [oracle.encode(a, form) for a in (k, v)]
    held = [oracle.decode(*e, form) for e in enc]
    return (*(to_pool(c, form) for c, _ in enc), *(torch.from_numpy(s).cuda() for _, s in enc)), *held


def to_bf16(x):
    """float64 rounded once to the nearest bf16 (normal range), ties to even."""
    step = 2.0 ** (np.frexp(x)[1] - 8)
    return np.rint(x / step) * step


@pytest.mark.parametrize("form", ["bf16", "mxfp8", "mxfp4"])
def test_attention_weights_keep_their_digits(form):
    """Two tokens, the heavier one's value zero: out = v w / (1 + w), w = e^-x.

    x is exact but for the rounding of scale log2 e and its product, so w is off by 2 U x + 2 U (the exponential), at most
    8 U for x <= 3.  The three products of its terms round 3 U at most, 1 + w U, its reciprocal 2 U, the last product U:
    15 U in all.  The one rounding to bf16 may go either way only within that of a border."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    g = np.random.default_rng(21)
    B, Hq, Hk, d, page = 40, 16, 2, 64, 16
    k, v = np.zeros((B, Hk, page, d)), np.zeros((B, Hk, page, d))
    k[:, :, 0, 0], k[:, :, 1, 0] = 1, -1
    v[:, :, 1] = g.standard_normal((B, Hk, d))
    cache, _, held = cache_of(k, v, form)
    x = g.integers(1, 193, (B, Hq)) / 16.0
    q = torch.zeros((B, Hq, d), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = torch.from_numpy(x).cuda()
    y = gdn.attention_step(q, cache, i32(np.arange(B)[:, None]), i32([2] * B), scale=0.125)
    w = np.exp(-2 * 0.125 * n(q)[..., 0])[..., None]
    want = np.repeat(held[:, :, 1], Hq // Hk, 1) * w / (1 + w)
    lo, hi = (to_bf16(want * (1 + s * 15 * U)) for s in (-1, 1))
    got = n(y)
    off = (got < np.minimum(lo, hi)) | (got > np.maximum(lo, hi))
    assert not off.any(), f"{off.sum()} of {off.size} outputs are not the nearest"
