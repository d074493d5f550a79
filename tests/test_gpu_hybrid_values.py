"""What a new token's attention makes of its weights and of values at the ends of
the number formats, on the GPU: the weights' digits, far and infinite values,
blocks whose scale is NaN or the least there is, queries beyond 16 bits' range,
long sums in fp32."""
import numpy as np
import pytest

import hybrid_oracle as oracle
from layer_oracle import U, check
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


def spread(B, L, Hk, page, d):
    """Pages of B sequences of up to L tokens, one after the other: (a table, k and v of zeros)."""
    width = -(-L // page)
    return np.arange(B * width).reshape(B, width), *(np.zeros((B * width, Hk, page, d)) for _ in range(2))


FAR = [(40, 2, 35), (40, 35, 2), (200, 7, 8), (200, 150, 149), (5000, 3, 4200), (5000, 4200, 3), (5000, 1000, 1001)]


@pytest.mark.parametrize("kind,form", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "mxfp8"), ("f32", "mxfp8"), ("bf16", "mxfp4")])
def test_attention_of_far_values_whose_weight_vanishes(kind, form):
    """A value near the type's end at a token whose weight is zero in 32 bits adds nothing, wherever the largest score
    lies: before it, behind it, in another wave or another run of tiles."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    rng = Rng(22)
    Hk, d, page = 2, 64, 64
    for L, top, far in FAR:
        table, k, v = spread(1, L, Hk, page, d)
        k[top // page, :, top % page, 0] = 18.75  # a score of 300 (288 in 8 or 4 bits): other weights are e^-288 at most
        v[top // page, :, top % page] = rng.g.integers(-3, 4, (Hk, d))
        v[far // page, :, far % page, ::2] = 1.75 * 2.0 ** 126
        cache, kk, vv = cache_of(k, v, form)
        q = torch.zeros((1, 4, d), dtype=_dtype(kind), device="cuda")
        q[..., 0] = 16
        lse = torch.empty((1, 4), device="cuda")
        y = gdn.attention_step(q, cache, i32(table), i32([L]), scale=1.0, lse=lse)
        want = np.repeat(vv[top // page, :, top % page], 2, 0)[None]  # one weight of exactly one
        check(n(y), want, np.zeros_like(want), kind, f"{L} {top} {far}")
        score = np.full((1, 4), 16 * kk[top // page, 0, top % page, 0])
        check(n(lse), score, 4 * U * score, "f32", "lse")  # (log2 e, its product, ln 2 and its product)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_attention_of_infinite_values_beside_far_scores(kind):
    """An infinite value's channel is infinite while its weight is above 2^-100 of the largest, and no number where it is
    smaller; the other channels are as ever."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    rng = Rng(23)
    Hk, d, page, c = 2, 64, 64, 9
    for L, top, far in FAR:
        for score in (40.0, 300.0):  # weights of e^-40 = 2^-58 and of zero in 32 bits
            table, k, v = spread(1, L, Hk, page, d)
            v[:] = rng.g.standard_normal(v.shape)
            k[top // page, :, top % page, 0] = score / 16
            v[far // page, 0, far % page, c] = np.inf
            v[far // page, 1, far % page, c] = -np.inf
            cache, kk, vv = cache_of(k, v, kind)
            q = torch.zeros((1, 2, d), dtype=_dtype(kind), device="cuda")
            q[..., 0] = 16
            y = n(gdn.attention_step(q, cache, i32(table), i32([L]), scale=1.0))[0]
            if score == 40.0:
                assert np.isposinf(y[0, c]) and np.isneginf(y[1, c]), (L, top, far)
            else:
                assert not np.isfinite(y[:, c]).any() and not np.isneginf(y[0, c]) and not np.isposinf(y[1, c])
            rest = np.delete(np.arange(d), c)
            for h in range(Hk):
                rows = vv[:, h].reshape(-1, d)[:L][:, rest]
                (o, oe), _ = oracle.attend(n(q)[0, h: h + 1, :1], kk[:, h].reshape(-1, d)[:L, :1], rows, 1.0, False)
                check(y[h: h + 1, rest], o, oe, kind, f"{L} {top} {far} {score}")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("L", [3, 200, 5000])
def test_attention_of_infinite_values_without_a_weight(kind, L):
    """Every score minus infinity: zero, infinite values or not."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    table, k, v = spread(2, L, 1, 32, 64)
    k[..., 0] = -np.inf
    v[..., 3], v[..., 4] = np.inf, -np.inf
    cache, _, _ = cache_of(k, v, kind)
    q = torch.ones((2, 2, 64), dtype=_dtype(kind), device="cuda")
    lse = torch.empty((2, 2), device="cuda")
    y = gdn.attention_step(q, cache, i32(table), i32([L, L // 2]), lse=lse)
    assert not n(y).any() and np.isneginf(n(lse)).all()


MX = [("bf16", "mxfp8"), ("f32", "mxfp8"), ("bf16", "mxfp4"), ("f32", "mxfp4")]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind,form", MX)
def test_attention_of_visible_blocks_that_are_nan(kind, form, d):
    """Scale byte 255 in a key makes the rows that see it NaN, in a value its 32 channels; whatever the codes are."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    rng = Rng(24)
    B, L, Hk, page = 8, 150, 2, 64
    table, k, v = spread(B, L, Hk, page, d)
    k[:], v[:] = rng.g.standard_normal(k.shape), rng.g.standard_normal(v.shape)
    k[0, 0, 5], v[3, 0, 5] = 0, 0  # codes of zero
    cache, kk, vv = cache_of(k, v, form)
    blocks = [0, d // 32 - 1, 1, 0]
    bad = [(b, [5, 17, 70, 149][b % 4], blocks[b % 4]) for b in range(B)]  # sequence, position, block; head 0
    for b, at, block in bad:
        cache[2 if b < 4 else 3][table[b, at // page], 0, at % page, block] = 255
    q = rng.t(B, 4, d, kind=kind)
    lse = torch.empty((B, 4), device="cuda")
    y, lse_ = n(gdn.attention_step(q, cache, i32(table), i32([L] * B), lse=lse)), n(lse)
    for b, at, block in bad:
        nan = np.zeros((4, d), bool)
        nan[:2, slice(None) if b < 4 else slice(32 * block, 32 * block + 32)] = True
        assert np.array_equal(np.isnan(y[b]), nan), (b, at, block)
        assert np.array_equal(np.isnan(lse_[b]), [b < 4, b < 4, False, False])
        for h in range(2):
            rows = [a[table[b], h].reshape(-1, d)[:L] for a in (kk, vv)]
            (o, oe), _ = oracle.attend(n(q)[b, 2 * h: 2 * h + 2], *rows, d ** -0.5, False)
            keep = ~nan[2 * h: 2 * h + 2]
            check(y[b, 2 * h: 2 * h + 2][keep], o[keep], oe[keep], kind, f"{b} {h}")
    gk, gv = gdn.kv_read(cache, i32(table), L)
    assert np.isnan(n(gk)).sum() == np.isnan(n(gv)).sum() == 4 * 32


@pytest.mark.parametrize("kind,form", MX)
def test_blocks_of_the_least_scales(kind, form):
    """Scale bytes 0 to 16, which kv_write does not choose: 2^-127 to 2^-111."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    d, page = 64, 32
    codes = np.zeros((1, 1, page, d), np.uint8)
    top = {"mxfp8": 126, "mxfp4": 7}[form]  # 448, 6
    codes[0, 0, :, 0] = top
    codes[0, 0, :, 1:32] = np.arange(1, 32) * (4 if form == "mxfp8" else 1) % (top + 1)
    codes[0, 0, :, 32] = top
    scales = np.full((1, 1, page, 2), 127, np.uint8)
    scales[0, 0, :, 0] = np.arange(page) % 17
    pool = to_pool(codes, form)
    cache = (pool, pool, *(torch.from_numpy(scales).cuda() for _ in range(2)))
    want = oracle.decode(codes, scales, form)[0, 0]
    for dtype in (torch.float32, torch.bfloat16):
        got = gdn.kv_read(cache, i32([[0]]), page, dtype=dtype)
        for t in got:
            assert torch.equal(t[0, :, 0].cpu(), torch.from_numpy(want).to(dtype)), dtype  # (exact in fp32)
    # attention of the one token of each byte (a window of one): lse is its score, of ordinary size by query and scale
    q = torch.zeros((1, 1, d), dtype=_dtype(kind), device="cuda")
    q[..., 0] = 2.0 ** 120
    lse = torch.empty((1, 1), device="cuda")
    for s in range(page):
        scale = 2.0 ** -(s % 17)
        gdn.attention_step(q, cache, i32([[0]]), i32([s + 1]), scale=scale, window=1, lse=lse)
        x = scale * 2.0 ** 120 * want[s, 0]
        check(n(lse), np.array([[x]]), np.array([[8 * U * x]]), "f32", f"byte {s % 17}")


@pytest.mark.parametrize("form", ["mxfp8", "mxfp4"])
def test_attention_of_fp32_queries_beyond_16_bits(form):
    """Over quantised keys: infinite queries, and the largest finite one, which lies above the largest bf16 value."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    rng = Rng(25)
    L, d, page = 70, 64, 32
    table, k, v = spread(1, L, 1, page, d)
    k[:], v[:] = rng.g.standard_normal(k.shape), rng.g.standard_normal(v.shape)
    k[..., 0] = rng.g.choice([1.0, 2.0, 3.0], k.shape[:-1])
    k[..., 1] = rng.g.choice([-0.5, 0.25, 0.5], k.shape[:-1])
    cache, kk, vv = cache_of(k, v, form)
    keys, values = (a[table[0], 0].reshape(-1, d)[:L] for a in (kk, vv))
    assert keys[:, 0].min() > 0

    def attend(channel, value, scale):
        q = torch.zeros((1, 1, d), device="cuda")
        q[..., channel] = value
        lse = torch.empty((1, 1), device="cuda")
        y = gdn.attention_step(q, cache, i32(table), i32([L]), scale=scale, lse=lse)
        return n(q)[0], n(y)[0], n(lse)[0]

    for scale in (1.0, 2.0 ** -126):
        _, y, lse = attend(0, -float("inf"), scale)  # every score minus infinity
        assert not y.any() and np.isneginf(lse).all()
        _, y, lse = attend(0, float("inf"), scale)
        assert np.isnan(y).all() and np.isnan(lse).all()
    for sign in (1, -1):
        q, y, lse = attend(1, sign * torch.finfo(torch.float32).max, 2.0 ** -126)  # scores of up to 2
        (o, oe), (l, le) = oracle.attend(q[:, 1:2], keys[:, 1:2], values, 2.0 ** -126, False)
        check(y, o, oe, "f32", f"{sign}")
        check(lse, l, le, "f32", f"{sign}")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_fp32_scores_are_sums_of_four(d):
    """One product of 1 and d - 1 of 0.1255 of its last digit: a sum that adds them to the one loses each, or rounds each
    four of them up.  At most d / 4 meet it: off by no more than they are.  Then the scale, log2 e, ln 2 and three sums."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    term = 0.1255 * 2.0 ** -23
    for at in (0, 1, 5, d // 2 + 2, d - 1):
        k = torch.full((1, 1, 16, d), term, device="cuda")
        k[..., at] = 1
        lse = torch.empty((2, 1), device="cuda")
        gdn.attention_step(torch.ones((2, 1, d), device="cuda"), (k, k), i32([[0], [0]]), i32([1, 1]), scale=1.0, lse=lse)
        want = np.full((2, 1), 1 + (d - 1) * term)
        check(n(lse), want, np.full((2, 1), (d / 4) * term + 7 * U), "f32", f"{at}")
