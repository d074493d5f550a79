"""The paged cache, a new token's attention over it and the seam between two
blocks on the GPU, against the 64-bit oracle (hybrid_oracle.py) with its derived
bounds: types, formats, lengths from nothing to many tiles, odd sizes, strided
views, packed batches, missing pages, windows, garbage in places not visible."""
import numpy as np
import pytest

import hybrid_oracle as oracle
from layer_oracle import HALF_STEP, check
from test_gpu_layer import Rng, _dtype, _torch, n, offsets

pytestmark = pytest.mark.gpu

NAMES = {"bf16": "bfloat16", "f32": "float32", "mxfp8": "mxfp8", "mxfp4": "mxfp4"}


def i32(a):
    torch = _torch()
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def pool(rng, shape, form, kind, garbage=False):
    """(device pool, device scales or None, its values): random, or what no call may look at."""
    torch = _torch()
    if form in ("bf16", "f32"):
        t = rng.t(*shape, kind=form)
        if garbage:
            t = torch.full_like(t, float("nan"))
            t.view(-1)[::3] = float("inf")
        return t, None, n(t)
    if garbage:
        codes = rng.g.integers(0, 256 if form == "mxfp8" else 16, shape).astype(np.uint8)
        scales = np.full((*shape[:-1], shape[-1] // 32), 255, np.uint8)
    else:
        x = rng.g.standard_normal(shape) * np.exp(rng.g.standard_normal((*shape[:-1], 1)))
        codes, scales = oracle.encode(x, form)
    return to_pool(codes, form), torch.from_numpy(scales).cuda(), oracle.decode(codes, scales, form)


def to_pool(codes, form):
    torch = _torch()
    if form == "mxfp8":
        return torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)
    return torch.from_numpy(codes[..., 0::2] + 16 * codes[..., 1::2]).cuda()


def codes_of(t, form):
    torch = _torch()
    c = t.view(torch.uint8).cpu().numpy()
    return c if form == "mxfp8" else np.stack([c % 16, c // 16], -1).reshape(*c.shape[:-1], -1)


def tables(rng, lens, page, width=None, spare=2):
    """A table whose pages are shuffled, -1 where there is none; and the pool's pages."""
    used = [-(-x // page) for x in lens]
    pages = sum(used) + spare
    order = rng.g.permutation(pages)
    t = np.full((len(lens), width or max(max(used), 1)), -1, np.int32)
    at = 0
    for b, u in enumerate(used):
        t[b, :u] = order[at: at + u]
        at += u
    return t, pages


def place(table, pages, page, pos):
    """(page, row) of a position, or None."""
    if pos < 0 or pos // page >= len(table):
        return None
    p = table[pos // page]
    return (p, pos % page) if 0 <= p < pages else None


# ---- writing and reading ----

KV = [
    # kind, form, lens (packed) or (B, T), heads, d, page, starts, layout
    ("bf16", "bf16", (1, 1), 1, 64, 16, [0], "plain"),
    ("bf16", "bf16", (3, 1), 8, 128, 16, [5, 0, 100], "step"),
    ("f32", "f32", (2, 37), 3, 64, 32, [0, 16], "slices"),
    ("bf16", "mxfp8", (2, 100), 5, 128, 64, None, "plain"),
    ("f32", "mxfp8", (1, 33), 2, 256, 16, [31], "odd"),
    ("bf16", "mxfp4", (64, 1), 4, 128, 32, list(range(64)), "step"),
    ("f32", "mxfp4", (1, 300), 1, 64, 256, [1], "plain"),
    ("bf16", "bf16", [5, 0, 1, 130, 2, 0, 70], 6, 64, 16, [0, 3, 9, 15, 16, 17, 33], "slices"),
    ("bf16", "mxfp8", [64, 1, 0, 33], 2, 128, 32, [7, 0, 0, 1], "plain"),
    ("f32", "mxfp4", [1] * 90, 3, 64, 16, list(range(90)), "odd"),
    ("bf16", "bf16", [0, 0], 2, 64, 16, None, "plain"),
    ("bf16", "bf16", (2, 900), 16, 256, 1024, [0, 200], "odd"),
]


def _rows(rng, lead, heads, d, kind, layout):
    torch = _torch()
    if layout == "slices":  # of one projection's rows
        return rng.t(*lead, 3 * heads, d, kind=kind)[..., heads: 2 * heads, :]
    if layout == "odd":  # off 16 bytes
        x = rng.t(*lead, heads, d, kind=kind)
        flat = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:]
        return flat.copy_(x.view(-1)).view(x.shape)
    return rng.t(*lead, heads, d, kind=kind)


@pytest.mark.parametrize("kind,form,lens,heads,d,page,starts,layout", KV)
def test_write_and_read(kind, form, lens, heads, d, page, starts, layout):
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    rng = Rng(1000 * heads + d + page)
    packed = isinstance(lens, list)
    each = lens if packed else [lens[1]] * lens[0]
    B, total = len(each), sum(each)
    T = total + 3 if packed else lens[1]  # (three rows behind the last sequence)
    lead = (T,) if packed else (B,) if layout == "step" else (B, T)
    k, v = _rows(rng, lead, heads, d, kind, layout), _rows(rng, lead, heads, d, kind, layout)
    with torch.no_grad():  # blocks of zeros, far magnitudes and ties
        for x in (k, v):
            if x.shape[0] > 1:
                x[0, ..., :32] = 0
                x[1] *= 2.0 ** -100
            x[-1, ..., -1] *= 1000
    at = [0] * B if starts is None else starts
    table, pages = tables(rng, [a + m for a, m in zip(at, each)], page)
    ks, vs = [pool(rng, (pages, heads, page, d), form, kind) for _ in range(2)]
    cache = (ks[0], vs[0]) if ks[1] is None else (ks[0], vs[0], ks[1], vs[1])
    off = offsets(each) if packed else None
    start = None if starts is None else i32(starts)
    before = [t.clone().view(torch.uint8) for t in cache]
    gdn.kv_write(k, v, cache, i32(table), start, seq_offsets=off)
    torch.cuda.synchronize()
    firsts = np.concatenate([[0], np.cumsum(each)])
    want_rows = []
    for x, p, s, old, olds in ((k, ks[0], ks[1], before[0], before[2] if ks[1] is not None else None),
                               (v, vs[0], vs[1], before[1], before[3] if ks[1] is not None else None)):
        rows = n(x).reshape(-1, heads, d)
        held = np.zeros((pages, page), bool)
        for b in range(B):
            for t in range(each[b]):
                held[place(table[b], pages, page, at[b] + t)] = True
        src = np.concatenate([np.arange(firsts[b], firsts[b + 1]) for b in range(B)]).astype(int)
        dst = [place(table[b], pages, page, at[b] + t) for b in range(B) for t in range(each[b])]
        pg, rw = np.array([x[0] for x in dst], int), np.array([x[1] for x in dst], int)
        if s is None:
            got = n(p)
            assert np.array_equal(got[pg, :, rw], rows[src])
            want_rows.append(rows[src])
        else:
            codes, scales = oracle.encode(rows[src], form)
            assert np.array_equal(s.cpu().numpy()[pg, :, rw], scales)
            c = codes_of(p, form)[pg, :, rw]
            table_, sign = oracle.TABLE[form], 128 if form == "mxfp8" else 8
            assert np.array_equal(table_[c % sign], table_[codes % sign])
            assert np.array_equal((c >= sign)[table_[c % sign] != 0], (codes >= sign)[table_[c % sign] != 0])
            assert np.array_equal(s.cpu().numpy().transpose(0, 2, 1, 3)[~held],
                                  olds.cpu().numpy().reshape(s.shape).transpose(0, 2, 1, 3)[~held])
            want_rows.append(oracle.decode(codes, scales, form))
        now, was = p.view(torch.uint8).cpu().numpy(), old.cpu().numpy().reshape(p.view(torch.uint8).shape)
        assert np.array_equal(now.transpose(0, 2, 1, 3)[~held], was.transpose(0, 2, 1, 3)[~held])
    # back out, in both types where the cache is quantised
    for dtype in ([None] if ks[1] is None else [None, torch.float32, torch.bfloat16]):
        gk, gv = gdn.kv_read(cache, i32(table), T, start, seq_offsets=off, dtype=dtype)
        for g, w in zip((gk, gv), want_rows):
            assert g.dtype == (dtype or (_dtype(form) if ks[1] is None else torch.bfloat16))
            got = n(g).reshape(-1, heads, d)
            assert np.array_equal(got[:total] if packed else got, w)  # exact: codes times powers of two
            assert not packed or not got[total:].any()


def test_write_and_read_leave_rows_without_a_place():
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    rng = Rng(5)
    k, v = rng.t(2, 40, 2, 64, kind="bf16"), rng.t(2, 40, 2, 64, kind="bf16")
    table = np.array([[1, -1, 0], [7, 3, 2 ** 31 - 1]], np.int32)  # pages 0..3: sequence 0 lacks one, sequence 1 has only its second
    cache = gdn.kv_cache(4, 2, 16, 64)
    gdn.kv_write(k, v, cache, i32(table), i32([-2, 20]))
    torch.cuda.synchronize()
    want = np.zeros((4, 2, 16, 64))
    kk = n(k)
    for b, s in ((0, -2), (1, 20)):
        for t in range(40):
            at = place(table[b], 4, 16, s + t)
            if at:
                want[at[0], :, at[1]] = kk[b, t]
    assert np.array_equal(n(cache.k), want) and want[0].any() and want[3].any() and not want[2].any()
    outs = [torch.full((2, 40, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gdn.kv_read(cache, i32(table), 40, i32([-2, 20]), k_out=outs[0], v_out=outs[1])
    fresh, _ = gdn.kv_read(cache, i32(table), 40, i32([-2, 20]))
    for b, s in ((0, -2), (1, 20)):
        for t in range(40):
            there = place(table[b], 4, 16, s + t) is not None
            assert np.array_equal(n(outs[0])[b, t], kk[b, t] if there else np.full((2, 64), 9.0))
            assert np.array_equal(n(fresh)[b, t], kk[b, t] if there else np.zeros((2, 64)))


@pytest.mark.parametrize("form", ["mxfp8", "mxfp4"])
def test_every_code_and_every_tie(form):
    """Blocks that hold every code, the values half-way between neighbours and just beside them, at several scales."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    t = oracle.TABLE[form]
    mid = (t[1:] + t[:-1]) / 2
    x = np.concatenate([t, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    x = np.concatenate([x, -x])
    x = np.concatenate([x, np.zeros(-len(x) % 62)]).reshape(-1, 62)
    x = np.concatenate([x, np.full((len(x), 2), t[-1])], 1)[:, [*range(31), 62, *range(31, 62), 63]]  # the largest in every block
    x = np.concatenate([x * 2.0 ** s for s in (0, 1, -7, 60, -100)])
    rows = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()[:, None]
    cache = gdn.kv_cache(-(-len(x) // 16), 1, 16, 64, form)
    table = i32(np.arange(-(-len(x) // 16))[None])
    gdn.kv_write(rows[None], rows[None], cache, table)
    codes, scales = oracle.encode(np.asarray(rows.cpu(), np.float64), form)
    got = gdn.kv_read(cache, table, len(x), dtype=torch.float32)[0]
    assert np.array_equal(n(got)[0], oracle.decode(codes, scales, form))


@pytest.mark.parametrize("form", ["mxfp8", "mxfp4"])
def test_infinities_and_nan_make_their_block_nan(form):
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    rng = Rng(8)
    k = rng.t(1, 16, 1, 64)
    k[0, 3, 0, 5], k[0, 4, 0, 40], k[0, 5, 0, 0] = float("nan"), float("inf"), -float("inf")
    cache = gdn.kv_cache(1, 1, 16, 64, form)
    gdn.kv_write(k, k, cache, i32([[0]]))
    for dtype in (torch.float32, torch.bfloat16):
        got = n(gdn.kv_read(cache, i32([[0]]), 16, dtype=dtype)[0])[0, :, 0]
        bad = np.zeros((16, 64), bool)
        bad[3, :32] = bad[4, 32:] = bad[5, :32] = True
        assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


# ---- attention ----

ATTEND = [
    # kind, form, lens, Hq, Hk, d, page, window, sinks
    ("bf16", "bf16", [1], 1, 1, 64, 16, 0, 0),
    ("bf16", "bf16", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129], 4, 2, 128, 16, 0, 0),
    ("f32", "f32", [0, 1, 15, 16, 17, 33, 100, 257], 6, 2, 64, 16, 0, 0),
    ("bf16", "mxfp8", [5, 0, 64, 300], 8, 1, 128, 64, 0, 0),
    ("f32", "mxfp8", [33, 1, 95], 3, 3, 128, 32, 0, 0),
    ("bf16", "mxfp4", [77, 200, 16, 31], 5, 1, 64, 32, 0, 0),
    ("f32", "mxfp4", [40, 41], 2, 2, 256, 16, 0, 0),
    ("bf16", "bf16", [700, 3, 259], 16, 1, 256, 128, 0, 0),
    ("f32", "f32", [130, 64], 4, 4, 256, 64, 0, 0),
    ("bf16", "bf16", [90, 500], 17, 1, 128, 16, 0, 0),       # more query heads than a tile of 16
    ("bf16", "mxfp8", [90, 333], 48, 1, 64, 32, 0, 0),
    ("f32", "f32", [65, 33], 40, 2, 64, 16, 0, 0),
    ("bf16", "bf16", [1, 50, 400, 1000], 8, 2, 64, 16, 100, 0),
    ("f32", "f32", [10, 333, 64, 2000], 4, 2, 64, 32, 33, 7),
    ("bf16", "mxfp8", [700, 90, 96, 97], 4, 4, 128, 16, 64, 32),
    ("bf16", "mxfp4", [1500, 2], 8, 8, 128, 1024, 1, 1),
    ("f32", "mxfp8", [600], 2, 1, 64, 64, 500, 90),
    ("bf16", "bf16", [1500], 8, 4, 128, 64, 1490, 100),      # sinks that meet the window
    ("bf16", "bf16", [9001, 4], 12, 12, 128, 64, 0, 0),
    ("f32", "f32", [5000], 4, 1, 128, 256, 0, 0),
    ("bf16", "mxfp8", [20011], 32, 8, 128, 64, 0, 0),
    ("bf16", "mxfp4", [7000, 100, 3000], 8, 2, 256, 16, 0, 0),
    ("bf16", "bf16", [37] * 300, 2, 1, 64, 16, 0, 0),        # more sequences than a wave has lanes
    ("bf16", "bf16", [4000] + [3] * 70, 4, 2, 64, 32, 0, 0),
]
# many sequences, none cut: with few tiles, up to 32, and more than 32
ATTEND += [(kind, form, lens, Hq, Hk, d, page, window, 0)
           for kind, form, Hq, Hk, d, page in [("bf16", "bf16", 8, 4, 128, 16), ("f32", "f32", 16, 8, 64, 32),
                                               ("bf16", "mxfp8", 34, 2, 128, 64), ("f32", "mxfp4", 6, 6, 64, 16)]
           for lens, window in [([2, 0, 63, 128] * 20, 0), ([300, 1, 129, 0, 1000] * 16, 90), ([33, 500] * 35, 0),
                                ([0, 1100, 700, 20] * 15, 0)]]


def _attention_case(kind, form, lens, Hq, Hk, d, page, window, sinks, seed, width=None):
    """(q, cache, table, lens, values of k, of v): what is not visible holds garbage."""
    torch = _torch()
    rng = Rng(seed)
    table, pages = tables(rng, lens, page, width)
    k, v = [pool(rng, (pages, Hk, page, d), form, kind) for _ in range(2)]
    bad = pool(rng, (pages, Hk, page, d), form, kind, garbage=True)
    seen = np.zeros((pages, page), bool)
    for b, length in enumerate(lens):
        for p in oracle.visible(length, table.shape[1] * page, window, sinks):
            at = place(table[b], pages, page, p)
            if at:
                seen[at] = True
    hide = torch.from_numpy(~seen).cuda()
    for t in (k, v):
        t[0].view(torch.uint8).transpose(1, 2)[hide] = bad[0].view(torch.uint8).transpose(1, 2)[hide]
        if t[1] is not None:
            t[1].transpose(1, 2)[hide] = bad[1].transpose(1, 2)[hide]
    q = rng.t(len(lens), Hq, d, kind=kind, scale=1.5)
    cache = (k[0], v[0]) if k[1] is None else (k[0], v[0], k[1], v[1])
    return q, cache, table, k[2], v[2]


def _expect(q, table, lens, kv, vv, scale, window, sinks, kind):
    """(out, bound), (lse, bound) over the batch."""
    B, Hq, d = q.shape
    pages, Hk, page, _ = kv.shape
    o, oe, l, le = np.zeros((B, Hq, d)), np.zeros((B, Hq, d)), np.zeros((B, Hq)), np.zeros((B, Hq))
    qq, G = n(q), Hq // Hk
    for b in range(B):
        at = [place(table[b], pages, page, p) for p in oracle.visible(lens[b], table.shape[1] * page, window, sinks)]
        at = [x for x in at if x]
        pg, rw = np.array([x[0] for x in at], int), np.array([x[1] for x in at], int)
        for h in range(Hk):
            g = slice(h * G, (h + 1) * G)
            (o[b, g], oe[b, g]), (l[b, g], le[b, g]) = oracle.attend(qq[b, g], kv[pg, h, rw], vv[pg, h, rw], scale, kind == "bf16")
    return (o, oe), (l, le)


def _check_attention(y, lse, want, kind, what=""):
    (o, oe), (l, le) = want
    check(n(y), o, oe, kind, what + " out")
    got, none = n(lse), np.isneginf(l)
    assert np.array_equal(np.isneginf(got), none)
    check(np.where(none, 0, got), np.where(none, 0, l), le, "f32", what + " lse")


@pytest.mark.parametrize("kind,form,lens,Hq,Hk,d,page,window,sinks", ATTEND)
def test_attention(kind, form, lens, Hq, Hk, d, page, window, sinks):
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    q, cache, table, kv, vv = _attention_case(kind, form, lens, Hq, Hk, d, page, window, sinks, len(lens) * 7 + d)
    lse = torch.full((len(lens), Hq), float("nan"), device="cuda")
    y = gdn.attention_step(q, cache, i32(table), i32(lens), window=window, sinks=sinks, lse=lse)
    torch.cuda.synchronize()
    assert y.dtype == q.dtype and y.shape == q.shape
    _check_attention(y, lse, _expect(q, table, lens, kv, vv, d ** -0.5, window, sinks, kind), kind)


def test_attention_lengths_beyond_the_table_and_missing_pages():
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    lens = [100, 64, 200, 40]
    q, cache, table, kv, vv = _attention_case("bf16", "bf16", lens, 4, 2, 64, 16, 0, 0, 3)
    table[0, 2], table[2, 0], table[2, 5], table[3, :] = -1, 2 ** 31 - 1, len(kv), -7  # no pages there
    given = [100, 2 ** 31 - 1, 2 ** 31 - 1, -5]
    table[1, 4:] = -1
    lse = torch.empty((4, 4), device="cuda")
    # sequence 2: the table's reach; what lies behind its 200 tokens in its last page is garbage
    given[2] = 200
    y = gdn.attention_step(q, cache, i32(table), i32(given), lse=lse)
    want = _expect(q, table, [100, 64, 200, 0], kv, vv, 0.125, 0, 0, "bf16")
    _check_attention(y, lse, want, "bf16")
    assert not n(y)[3].any()


@pytest.mark.parametrize("form", ["bf16", "mxfp8"])
def test_attention_of_strided_rows_with_a_scale(form):
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    lens = [70, 300, 5]
    q, cache, table, kv, vv = _attention_case("bf16", form, lens, 6, 2, 128, 32, 0, 0, 9)
    rows = torch.zeros(3, 9, 129, dtype=torch.bfloat16, device="cuda")  # off 16 bytes
    rows[:, 2:8, 1:] = q
    out = torch.full((6, 3, 140), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)  # heads outermost
    y = gdn.attention_step(rows[:, 2:8, 1:], cache, i32(table), i32(lens), scale=-0.3, out=out[..., 3:131])
    assert y.data_ptr() == out[..., 3:131].data_ptr()
    (o, oe), _ = _expect(q, table, lens, kv, vv, -0.3, 0, 0, "bf16")
    check(n(y), o, oe, "bf16")
    assert (n(out)[..., :3] == 7).all() and (n(out)[..., 131:] == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_attention_of_far_scores(kind):
    """Scores in the hundreds, the largest first or last: the running maximum moves, weights underflow."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    lens = [500, 130]
    q, cache, table, kv, vv = _attention_case(kind, kind, lens, 2, 1, 64, 16, 0, 0, 4)
    for b, at in ((0, 3), (1, 129)):
        pg, rw = place(table[b], len(kv), 16, at)
        cache[0][pg, 0, rw] = q[b, 0] * 4
    kv = n(cache[0])
    lse = torch.empty((2, 2), device="cuda")
    y = gdn.attention_step(q, cache, i32(table), i32(lens), scale=2.0, lse=lse)
    _check_attention(y, lse, _expect(q, table, lens, kv, vv, 2.0, 0, 0, kind), kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_attention_of_nan_and_infinite_tokens(kind):
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    lens = [50, 50, 50, 50, 1]
    q, cache, table, kv, vv = _attention_case(kind, kind, lens, 2, 1, 64, 16, 0, 0, 6)
    at = [place(table[b], len(kv), 16, 20) for b in range(4)]
    cache[0][at[0][0], 0, at[0][1]] = float("nan")      # a key: the whole row is NaN
    cache[1][at[1][0], 0, at[1][1], 5] = float("nan")   # a value: its channel
    cache[1][at[2][0], 0, at[2][1], 7] = float("inf")
    cache[1][at[2][0], 0, at[2][1], 8] = -float("inf")
    cache[0][at[3][0], 0, at[3][1]] = 0                 # a key of minus infinity's score: weight zero
    cache[0][at[3][0], 0, at[3][1], 0] = -float("inf")
    cache[1][table[4, 0], 0, 0, 9] = float("inf")       # a weight of exactly one
    q[:, :, 0] = q[:, :, 0].abs() + 0.1
    lse = torch.empty((5, 2), device="cuda")
    y = gdn.attention_step(q, cache, i32(table), i32(lens), lse=lse)
    got = n(y)
    assert np.isnan(got[0]).all() and np.isnan(n(lse)[0]).all()
    assert np.isnan(got[1, :, 5]).all() and np.isfinite(np.delete(got[1], 5, 1)).all()
    assert np.isposinf(got[2, :, 7]).all() and np.isneginf(got[2, :, 8]).all()
    assert np.isfinite(np.delete(got[2], [7, 8], 1)).all()
    assert np.isposinf(got[4, :, 9]).all() and np.isfinite(np.delete(got[4], 9, 1)).all()
    kk, vals = n(cache[0]), n(cache[1])
    keep = [p for p in range(50) if p != 20]
    pg = np.array([table[3, p // 16] for p in keep])
    rw = np.array([p % 16 for p in keep])
    (o, oe), (l, le) = oracle.attend(n(q)[3], kk[pg, 0, rw], vals[pg, 0, rw], 0.125, kind == "bf16")
    check(got[3], o, oe, kind)
    check(n(lse)[3], l, le, "f32")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_attention_of_scores_that_are_all_minus_infinity(kind):
    """The sum of weights is zero, as where nothing is visible."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    q, cache, table, kv, vv = _attention_case(kind, kind, [40, 3], 2, 1, 64, 16, 0, 0, 6)
    cache[0].zero_()
    cache[0][..., 0] = -float("inf")
    q[:, :, 0] = 1
    lse = torch.empty((2, 2), device="cuda")
    y = gdn.attention_step(q, cache, i32(table), i32([40, 3]), lse=lse)
    assert not n(y).any() and np.isneginf(n(lse)).all()


def test_attention_of_a_pool_beyond_4_gib():
    """Rows whose offset in the pool passes 32 bits."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    page, d = 1024, 256
    pages = (1 << 32) // (page * d * 2) + 40  # 4 GiB and a little
    pools = [torch.zeros((pages, 1, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rng = Rng(12)
    table = np.array([[pages - 1, 3, pages - 30]], np.int32)
    k, v = rng.t(1, 2500, 1, d, kind="bf16"), rng.t(1, 2500, 1, d, kind="bf16")
    gdn.kv_write(k, v, pools, i32(table))
    q = rng.t(1, 4, d, kind="bf16")
    lse = torch.empty((1, 4), device="cuda")
    y = gdn.attention_step(q, pools, i32(table), i32([2500]), lse=lse)
    (o, oe), (l, le) = oracle.attend(n(q)[0], n(k)[0, :, 0], n(v)[0, :, 0], 1 / 16, True)
    check(n(y)[0], o, oe, "bf16")
    check(n(lse)[0], l, le, "f32")
    back, _ = gdn.kv_read(pools, i32(table), 2500)
    assert torch.equal(back, k)


# ---- the seam ----

SEAM = [
    # kind, lens (packed) or (B, T) or (B,) for a token each, D, y, gate, post, weight, alpha, layout
    ("bf16", (1, 1), 8, True, "channel", True, True, 1.0, "plain"),
    ("f32", (1, 1), 1, True, None, True, True, 1.0, "plain"),
    ("bf16", (2, 3), 64, True, "sequence", False, True, 1.0, "plain"),
    ("f32", (3, 50), 100, True, "sequence", True, True, 0.5, "slices"),
    ("bf16", (2, 37), 512, True, "channel", True, False, 1.0, "plain"),
    ("bf16", (1, 65), 520, True, None, True, True, -1.5, "odd"),
    ("f32", (2, 40), 1001, True, "sequence", False, True, 1.0, "plain"),
    ("bf16", (70,), 1024, True, "sequence", True, True, 1.0, "plain"),
    ("bf16", (5, 9), 2048, True, "sequence", True, True, 1.0, "slices"),
    ("f32", (2, 33), 2047, True, "channel", True, True, 1.0, "plain"),
    ("bf16", (64,), 4096, True, "channel", False, True, 1.0, "plain"),
    ("f32", (3, 7), 4100, True, "channel", True, True, 2.0, "plain"),
    ("bf16", (1, 21), 8192, True, "sequence", True, True, 1.0, "plain"),
    ("bf16", (2, 5), 16384, True, "channel", True, True, 1.0, "plain"),
    ("f32", (1, 4), 16383, True, "sequence", True, True, 1.0, "odd"),
    ("bf16", (2, 30), 256, False, None, False, True, 1.0, "plain"),
    ("f32", (2, 30), 256, False, None, False, True, 0.7, "plain"),
    ("bf16", [5, 0, 1, 130, 2, 0, 70], 96, True, "sequence", True, True, 1.0, "plain"),
    ("f32", [0, 0, 3], 33, True, "sequence", False, True, 1.0, "plain"),
    ("bf16", [1] * 90, 2056, True, "sequence", True, True, 1.0, "plain"),
    ("f32", [700, 3, 900], 64, True, "channel", True, True, 1.0, "slices"),
    ("bf16", (1, 5000), 128, True, "sequence", True, True, 1.0, "plain"),
    ("bf16", [3000, 1500], 1100, True, "sequence", True, True, 1.0, "odd"),
    ("bf16", (2, 0), 64, True, "sequence", True, True, 1.0, "plain"),
]
# rows off 16 bytes and of no whole vectors, in every kernel's widths: the last vector of a row is moved back into it
SEAM += [(kind, lens, D, True, gate, True, True, 1.0, layout)
         for D in [1, 2, 3, 4, 5, 7, 9, 63, 65, 67, 127, 129, 150, 250, 257, 501, 1001, 1025, 2001, 4003, 7001, 9001]
         for kind, lens, gate, layout in [("bf16", (2, 19), "sequence", "plain"), ("f32", [5, 0, 31, 1], "sequence", "odd")]]
SEAM += [("bf16", [200, 0, 33, 1], 64, True, "sequence", True, True, 1.0, "odd"),
         ("bf16", [200, 0, 33, 1], 128, True, "sequence", False, True, 1.0, "slices"),
         ("bf16", [200, 0, 33, 1], 256, True, "sequence", True, True, 1.0, "plain"),
         ("f32", (3, 90), 128, True, "channel", True, True, 1.0, "plain"),
         ("bf16", (1, 9000), 64, True, "channel", True, True, 1.0, "plain")]


class SeamCase:
    def __init__(self, kind, lens, D, has_y, gate, post, weight, alpha, layout, eps=1e-6):
        torch = _torch()
        rng = Rng(D + len(lens))
        self.packed = isinstance(lens, list)
        self.each = lens if self.packed else [1] * lens[0] if len(lens) == 1 else [lens[1]] * lens[0]
        self.total = sum(self.each)
        lead = (self.total + 2,) if self.packed else lens
        self.kind, self.D, self.alpha, self.eps = kind, D, alpha, eps

        def rows(scale=1.0):
            if layout == "slices":
                return rng.t(*lead, 3 * D, kind=kind, scale=scale)[..., D: 2 * D]
            x = rng.t(*lead, D, kind=kind, scale=scale)
            if layout == "odd":
                return torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].copy_(x.view(-1)).view(x.shape)
            return x

        self.x, self.y = rows(2.0), rows() if has_y else None
        B = len(self.each)
        self.gate = None if gate is None else rng.t(*((B, D) if gate == "sequence" else (D,)), scale=0.5, mean=0.3)
        self.post = rng.t(D, scale=0.2, mean=1.0) if post else None
        self.weight = rng.t(D, scale=0.2, mean=1.0) if weight else None
        self.dh, self.dn = rows(), rows() if weight else None
        self.off = offsets(self.each) if self.packed else None
        self.firsts = np.concatenate([[0], np.cumsum(self.each)]).astype(int)

    def flat(self, t):
        return None if t is None else n(t).reshape(-1, self.D)[: self.total]

    def row_gate(self):
        g = n(self.gate)
        return np.repeat(g, self.each, 0) if g is not None and g.ndim == 2 else g

    def args(self):
        return dict(gate=self.gate, post_weight=self.post, weight=self.weight, residual_scale=self.alpha, eps=self.eps,
                    seq_offsets=self.off)

    def expect(self):
        return oracle.seam(self.flat(self.x), self.flat(self.y), self.row_gate(), n(self.post), n(self.weight), self.alpha,
                           self.eps)

    def expect_backward(self, dh=True):
        groups = None
        if self.gate is not None and self.gate.dim() == 2:
            groups = list(zip(self.firsts[:-1], self.firsts[1:]))
        return oracle.seam_backward(self.flat(self.dh) if dh else None, self.flat(self.dn), self.flat(self.x), self.flat(self.y),
                                    self.row_gate(), n(self.post), n(self.weight), self.alpha, self.eps, groups)


@pytest.mark.parametrize("kind,lens,D,has_y,gate,post,weight,alpha,layout", SEAM)
def test_residual_norm(kind, lens, D, has_y, gate, post, weight, alpha, layout):
    import gated_delta_rule_scan_amd as gdn

    c = SeamCase(kind, lens, D, has_y, gate, post, weight, alpha, layout)
    h, nn = gdn.residual_norm(c.x, c.y, **c.args())
    (eh, ehb), en = c.expect()
    if not has_y and alpha == 1.0:
        assert h is c.x
    else:
        check(c.flat(h), eh, ehb, kind, "h")
        assert h.dtype == c.x.dtype and not n(h).reshape(-1, D)[c.total:].any()
    assert (nn is None) == (not weight)
    if weight:
        check(c.flat(nn), *en, kind, "n")
        assert not n(nn).reshape(-1, D)[c.total:].any()


@pytest.mark.parametrize("kind,lens,D,has_y,gate,post,weight,alpha,layout", SEAM)
def test_residual_norm_backward(kind, lens, D, has_y, gate, post, weight, alpha, layout):
    import gated_delta_rule_scan_amd as gdn

    c = SeamCase(kind, lens, D, has_y, gate, post, weight, alpha, layout)
    got = dict(zip(("dx", "dy", "dgate", "dpost", "dweight"), gdn.residual_norm_backward(c.dh, c.dn, c.x, c.y, **c.args())))
    want = c.expect_backward()
    assert {k for k, v in got.items() if v is not None} == set(want)
    for k, (value, bound) in want.items():
        if k in ("dx", "dy"):
            check(c.flat(got[k]), value, bound, kind, k)
            assert got[k].dtype == c.x.dtype and not n(got[k]).reshape(-1, D)[c.total:].any()
        else:
            check(n(got[k]), value, bound, "f32", k)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_residual_norm_in_place_and_given_outputs(kind):
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    c = SeamCase(kind, [20, 0, 7], 200, True, "sequence", True, True, 1.0, "plain")
    h0, n0 = gdn.residual_norm(c.x, c.y, **c.args())
    g0 = gdn.residual_norm_backward(c.dh, c.dn, c.x, c.y, **c.args())
    x, dh = c.x.clone(), c.dh.clone()
    nout = torch.full_like(x, 5.0)
    h, nn = gdn.residual_norm(x, c.y, **c.args(), out=x, norm_out=nout)
    assert h.data_ptr() == x.data_ptr() and nn.data_ptr() == nout.data_ptr()
    assert torch.equal(h[:27], h0[:27]) and torch.equal(nn[:27], n0[:27])
    assert torch.equal(h[27:], c.x[27:]) and (nn[27:] == 5).all()  # rows of no sequence
    dy = torch.full_like(x, 5.0)
    g = gdn.residual_norm_backward(dh, c.dn, c.x, c.y, **c.args(), dx=dh, dy=dy)
    assert g[0].data_ptr() == dh.data_ptr()
    assert torch.equal(dh[:27], g0[0][:27]) and torch.equal(dy[:27], g0[1][:27])
    assert torch.equal(dh[27:], c.dh[27:]) and (dy[27:] == 5).all()
    assert all(torch.equal(a, b) for a, b in zip(g[2:], g0[2:]))
    # without dh, and without dn
    got = gdn.residual_norm_backward(None, c.dn, c.x, c.y, **c.args())
    want = c.expect_backward(dh=False)
    check(c.flat(got[0]), *want["dx"], kind, "dx")
    check(n(got[2]), *want["dgate"], "f32", "dgate")


@pytest.mark.parametrize("kind,D,layout", [("bf16", 2001, "plain"), ("bf16", 1100, "odd"), ("f32", 1027, "plain"), ("bf16", 4003, "plain"),
                                           ("f32", 8190, "odd"), ("bf16", 16381, "plain"), ("bf16", 1001, "plain"), ("f32", 67, "odd")])
@pytest.mark.parametrize("post,weight", [(False, False), (True, False), (False, True)])
def test_residual_norm_in_place_of_odd_widths(kind, D, layout, post, weight):
    """Rows of no whole vectors over several waves that do not wait for each other: no wave reads what another wrote."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    c = SeamCase(kind, (2, 400), D, True, "sequence", post, weight, 0.5, layout)
    h0, n0 = gdn.residual_norm(c.x, c.y, **c.args())
    g0 = gdn.residual_norm_backward(c.dh, c.dn, c.x, c.y, **c.args())
    (eh, ehb), _ = c.expect()
    check(c.flat(h0), eh, ehb, kind, "h")
    dh = c.dh.clone()
    gdn.residual_norm_backward(dh, c.dn, c.x, c.y, **c.args(), dx=dh)
    assert torch.equal(dh, g0[0])
    _, nn = gdn.residual_norm(c.x, c.y, **c.args(), out=c.x)
    assert torch.equal(c.x, h0) and (not weight or torch.equal(nn, n0))


def test_residual_norm_gradients_against_differences():
    """Directional differences of the forward call itself, in fp32."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    c = SeamCase("f32", (2, 6), 48, True, "sequence", True, True, 0.8, "plain")
    got = gdn.residual_norm_backward(c.dh, c.dn, c.x, c.y, **c.args())

    def loss(x, y, gate, post, weight):
        h, nn = gdn.residual_norm(x, y, gate, post, weight, 0.8)
        return float((h.double() * c.dh.double()).sum() + (nn.double() * c.dn.double()).sum())

    args = [c.x, c.y, c.gate, c.post, c.weight]
    step = 2.0 ** -6
    for i, (a, g) in enumerate(zip(args, got)):
        r = torch.randn(a.shape, generator=torch.Generator().manual_seed(i)).cuda()
        moved = lambda s: loss(*(a + s * r if j == i else b for j, b in enumerate(args)))
        # fourth order in the step: its error is of order step^4 times the fifth derivative
        slope = (8 * (moved(step) - moved(-step)) - (moved(2 * step) - moved(-2 * step))) / (12 * step)
        want = float((g.double() * r.double()).sum())
        scale = float((g.double() * r.double()).abs().sum())
        # 576 outputs, each off by up to 64 half steps of 2^-24 of values below 8, over a step of 2^-6: below 2e-2 if all
        # add up; a step of 2^-6 to the fourth is 6e-8
        assert abs(slope - want) <= 2e-3 * scale + 2e-2, (i, slope, want)
