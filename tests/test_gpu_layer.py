"""Short causal convolution, selective scan, rotary positions and the
single-token steps on the GPU, against the 64-bit oracle (layer_oracle.py) with
its derived bounds: types, layouts, lengths from nothing to many tiles, odd
sizes, strided views, packed batches with empty sequences, state slots."""
import numpy as np
import pytest

import layer_oracle as oracle

pytestmark = pytest.mark.gpu


def _torch():
    import torch

    return torch


def _dtype(kind):
    torch = _torch()
    return torch.bfloat16 if kind == "bf16" else torch.float32


class Rng:
    """Seeded device tensors in an operand's type, and the same values as float64 arrays."""

    def __init__(self, seed):
        self.g = np.random.default_rng(seed)

    def t(self, *shape, kind="f32", scale=1.0, mean=0.0):
        torch = _torch()
        a = torch.from_numpy((self.g.standard_normal(shape) * scale + mean).astype(np.float32))
        return a.to(_dtype(kind)).cuda()


def n(t):
    return None if t is None else t.detach().double().cpu().numpy()


def offsets(lens):
    torch = _torch()
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


# ---- short causal convolution ----

CONV = [
    # kind, lens (packed) or (B, T), D, W, act, bias, state
    ("bf16", (1, 1), 8, 4, "silu", True, True),
    ("bf16", (2, 2), 64, 4, "silu", True, True),       # fewer tokens than the history
    ("bf16", (3, 0), 64, 4, "none", False, True),      # no tokens: the state passes through
    ("f32", (1, 1560), 256, 4, "silu", True, True),
    ("bf16", (2, 259), 1001, 3, "silu", False, True),  # odd channels
    ("f32", (1, 77), 1, 2, "none", True, False),
    ("f32", (5, 33), 36, 3, "none", True, True),
    ("bf16", (1, 4097), 520, 2, "silu", False, False),
    ("bf16", (1, 9000), 4104, 4, "silu", True, True),   # several batches a run
    ("bf16", [5, 0, 1, 130, 2, 0, 700], 72, 4, "silu", True, True),
    ("f32", [0, 0], 16, 4, "silu", True, True),
    ("f32", [1] * 150, 33, 4, "silu", True, True),     # more sequences than a wave has lanes
    ("bf16", [64, 32, 96, 31, 33] * 30, 24, 3, "none", False, True),
    ("f32", [300], 128, 4, "silu", True, False),
]


@pytest.mark.parametrize("kind,lens,D,W,act,bias,state", CONV)
def test_conv(kind, lens, D, W, act, bias, state):
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(hash((D, W)) % 1000)
    packed = isinstance(lens, list)
    B = len(lens) if packed else lens[0]
    shape = (sum(lens), D) if packed else (*lens, D)
    x = r.t(*shape, kind=kind)
    w, b = r.t(D, W, scale=0.5), r.t(D) if bias else None
    s = r.t(B, W - 1, D, kind=kind) if state else None
    y, s2 = gdn.causal_conv(x, w, b, s, act, seq_offsets=offsets(lens) if packed else None)
    assert y.dtype == x.dtype and s2.dtype == x.dtype
    rows = np.split(n(x), np.cumsum(lens)[:-1]) if packed else list(n(x))
    outs = np.split(n(y), np.cumsum(lens)[:-1]) if packed else list(n(y))
    for i in range(B):
        s0 = n(s)[i] if state else np.zeros((W - 1, D))
        (want, err), last = oracle.conv(rows[i], n(w), n(b), s0, act == "silu")
        oracle.check(outs[i], want, err, kind, f"sequence {i}")
        assert np.array_equal(n(s2)[i], last), f"final state {i}"


def test_conv_views_slots_and_in_place():
    """x the second half of wider rows (odd offset, so rows are unaligned), out beside it in a wider buffer, states in
    a pool by index (one out of range), advanced in place; other slots and the rest of the buffer are untouched."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(5)
    B, T, D, W = 4, 41, 40, 4
    wide = r.t(B, T, 2 * D + 1, kind="bf16")
    x = wide[..., D + 1:]
    w = r.t(D, W)
    pool = r.t(9, W - 1, D, kind="bf16")
    before = pool.clone()
    index = torch.tensor([7, -1, 2, 9], dtype=torch.int32, device="cuda")
    buf = torch.full((B, T, 3 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    y, s2 = gdn.causal_conv(x, w, None, pool, "none", state_index=index, out=buf[..., D:2 * D], state_out=pool)
    assert s2 is pool and y.data_ptr() == buf[..., D:].data_ptr()
    assert (buf[..., :D] == 7).all() and (buf[..., 2 * D:] == 7).all()
    for i, slot in enumerate(index.tolist()):
        ok = 0 <= slot < 9
        s0 = n(before)[slot] if ok else np.zeros((W - 1, D))
        (want, err), last = oracle.conv(n(x)[i], n(w), None, s0, False)
        oracle.check(n(y)[i], want, err, "bf16", f"sequence {i}")
        if ok:
            assert np.array_equal(n(pool)[slot], last)
    rest = [i for i in range(9) if i not in (7, 2)]
    assert torch.equal(pool[rest], before[rest])


def test_conv_rows_behind_the_last_sequence_stay():
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(6)
    x = r.t(300, 64, kind="bf16")
    out = torch.full_like(x, 3.0)
    gdn.causal_conv(x, r.t(64, 4), seq_offsets=offsets([100, 57]), out=out)
    assert (out[157:] == 3).all() and not (out[:157] == 3).all()


def test_conv_offsets_out_of_range_are_clamped():
    """Offsets beyond the buffer, or falling: nothing outside the buffers is touched (guarded), nothing hangs."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(7)
    whole = torch.full((3, 300, 64), 3.0, device="cuda")
    out = whole[1]
    x, w = r.t(300, 64), r.t(64, 4)
    for off in ([0, 100, 2 ** 31 - 1], [-5, 100, 300], [250, 100, 280], [2 ** 31 - 1, -2 ** 31, 7]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        gdn.causal_conv(x, w, seq_offsets=o, out=out)
        gdn.selective_scan(x, x, -torch.ones(64, 4, device="cuda"), x[:, :4], x[:, :4], seq_offsets=o, out=out)
        torch.cuda.synchronize()
    assert (whole[0] == 3).all() and (whole[2] == 3).all()


@pytest.mark.parametrize("kind,B,D,W,act,bias", [("bf16", 64, 2048, 4, "silu", True), ("f32", 1, 7, 2, "none", False),
                                                 ("bf16", 3, 1001, 3, "silu", True), ("f32", 130, 40, 4, "silu", True)])
def test_conv_step(kind, B, D, W, act, bias):
    """Single tokens against the oracle; a row with no slot, its output and the other slots stay as they were."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(8)
    slots = B + 3
    pool = r.t(slots, W - 1, D, kind=kind)
    before = pool.clone()
    idx = r.g.permutation(slots)[:B].astype(np.int32)
    if B > 2:
        idx[1], idx[2] = -1, slots
    x, w, b = r.t(B, 2 * D, kind=kind)[:, D:], r.t(D, W, scale=0.5), r.t(D) if bias else None
    out = torch.full((B, D), 5.0, dtype=x.dtype, device="cuda")
    y = gdn.causal_conv_step(x, w, b, pool, act, torch.from_numpy(idx).cuda(), out=out)
    used = []
    for i, slot in enumerate(idx.tolist()):
        if not 0 <= slot < slots:
            assert (y[i] == 5).all()
            continue
        used.append(slot)
        (want, err), last = oracle.conv(n(x)[i: i + 1], n(w), n(b), n(before)[slot], act == "silu")
        oracle.check(n(y)[i: i + 1], want, err, kind, f"row {i}")
        assert np.array_equal(n(pool)[slot], last)
    rest = [i for i in range(slots) if i not in used]
    assert torch.equal(pool[rest], before[rest])


# ---- selective scan ----

SSM = [
    # kind, lens (packed) or (B, T), D, N, G, gate, skip, bias, softplus, state
    ("f32", (1, 1), 1, 1, 1, False, False, False, False, True),
    ("bf16", (2, 3), 8, 16, 1, True, True, True, True, True),
    ("f32", (1, 0), 8, 16, 1, True, True, True, True, True),
    ("f32", (1, 64), 5, 16, 1, True, True, True, True, False),
    ("bf16", (2, 257), 24, 16, 2, True, True, True, True, True),
    ("f32", (1, 1025), 12, 8, 1, False, True, True, True, True),
    ("f32", (1, 2500), 9, 3, 3, True, True, False, True, False),
    ("bf16", (1, 700), 20, 37, 1, True, False, True, True, True),
    ("f32", (3, 130), 16, 64, 4, True, True, True, True, True),
    ("f32", (1, 90), 3, 256, 1, False, False, True, True, True),
    ("bf16", [5, 0, 1, 300, 64, 0, 1100], 16, 16, 1, True, True, True, True, True),
    ("f32", [1] * 70, 4, 16, 1, True, True, True, True, True),
    ("f32", [17, 4, 255, 256, 3], 24, 16, 2, True, True, True, True, False),
    ("f32", [0, 0, 0], 8, 5, 1, False, False, False, True, True),
]


def _ssm_inputs(r, kind, lead, D, N, G, gate, skip, bias, softplus):
    torch = _torch()
    xz = r.t(*lead, 2 * D, kind=kind)
    bc = r.t(*lead, 2 * G * N + 3, kind=kind)
    kw = dict(x=xz[..., :D], dt=r.t(*lead, D, kind=kind, scale=0.5), A=-torch.exp(r.t(D, N, scale=0.7)),
              B=bc[..., 3: 3 + G * N].unflatten(-1, (G, N)), C=bc[..., 3 + G * N:].unflatten(-1, (G, N)),
              D=r.t(D) if skip else None, z=xz[..., D:] if gate else None,
              dt_bias=r.t(D, scale=2.0, mean=-3.0) if bias else None, dt_softplus=softplus)
    if not softplus:
        kw["dt"] = kw["dt"].abs() * 0.2
    return kw


def _ssm_oracle(kw, rows, state):
    take = lambda t: None if t is None else n(t)[rows]
    return oracle.ssm(take(kw["x"]), take(kw["dt"]), n(kw["A"]), take(kw["B"]), take(kw["C"]), n(kw["D"]), take(kw["z"]),
                      n(kw["dt_bias"]), kw["dt_softplus"], state)


@pytest.mark.parametrize("kind,lens,D,N,G,gate,skip,bias,softplus,state", SSM)
def test_selective_scan(kind, lens, D, N, G, gate, skip, bias, softplus, state):
    import gated_delta_rule_scan_amd as gdn

    r = Rng(D * 1000 + N)
    packed = isinstance(lens, list)
    B = len(lens) if packed else lens[0]
    kw = _ssm_inputs(r, kind, (sum(lens),) if packed else lens, D, N, G, gate, skip, bias, softplus)
    s = r.t(B, D, N) if state else None
    y, h = gdn.selective_scan(**kw, state_in=s, seq_offsets=offsets(lens) if packed else None)
    assert y.dtype == kw["x"].dtype and y.is_contiguous()
    at = np.concatenate([[0], np.cumsum(lens)]) if packed else None
    for i in range(B):
        rows = slice(at[i], at[i + 1]) if packed else i
        (want, err), (hw, he) = _ssm_oracle(kw, rows, n(s)[i] if state else np.zeros((D, N)))
        oracle.check(n(y)[rows], want, err, kind, f"sequence {i}")
        oracle.check(n(h)[i], hw, he, "f32", f"final state {i}")


@pytest.mark.parametrize("T", [36, 37, 40, 72, 73, 96, 97, 103, 104, 128, 129, 511, 512, 513])
@pytest.mark.parametrize("D,N,G", [(70, 16, 1), (200, 16, 2), (130, 33, 1), (65, 100, 1), (12, 256, 3)])
def test_selective_scan_around_chunk_borders(T, D, N, G):
    """Lengths on both sides of the split and of chunk, stage and load borders; channel tiles with a rest, groups that
    are no whole tile, entries over several waves."""
    import gated_delta_rule_scan_amd as gdn

    r = Rng(T * 7 + N)
    kw = _ssm_inputs(r, "f32", (1, T), D, N, G, True, True, True, True)
    s = r.t(1, D, N)
    y, h = gdn.selective_scan(**kw, state_in=s)
    (want, err), (hw, he) = _ssm_oracle(kw, 0, n(s)[0])
    oracle.check(n(y)[0], want, err, "f32", "out")
    oracle.check(n(h)[0], hw, he, "f32", "state")


@pytest.mark.parametrize("B,T,D,packed", [(1100, 75, 8, False), (2, 76, 33000, False), (90, 900, 6, True), (700, 5000, 3, True)])
def test_selective_scan_many_sequences_or_channels(B, T, D, packed):
    """Enough waves for one kernel, and packed batches of many sequences (one round of the search and several), a few
    sequences and channels of each against the oracle."""
    import gated_delta_rule_scan_amd as gdn

    r = Rng(B + T)
    lens = None
    if packed:
        cuts = np.sort(r.g.integers(0, T + 1, B - 1))
        lens = np.diff(np.concatenate([[0], cuts, [T]]))
    kw = _ssm_inputs(r, "bf16", (T,) if packed else (B, T), D, 16, 1, True, True, True, True)
    s = r.t(B, D, 16)
    y, h = gdn.selective_scan(**kw, state_in=s, seq_offsets=offsets(lens) if packed else None)
    at = np.concatenate([[0], np.cumsum(lens)]) if packed else None
    ch = np.unique(np.concatenate([r.g.integers(0, D, 4), [0, D - 1]]))
    cut = lambda t: t if t is None else t[..., ch]
    few = dict(kw, x=cut(kw["x"]), dt=cut(kw["dt"]), z=cut(kw["z"]), A=kw["A"][ch], D=cut(kw["D"]), dt_bias=cut(kw["dt_bias"]))
    seqs = np.unique(np.concatenate([r.g.integers(0, B, 6), [0, B - 1], [] if lens is None else [int(np.argmax(lens))]])).astype(int)
    for i in seqs:
        rows = slice(at[i], at[i + 1]) if packed else int(i)
        (want, err), (hw, he) = _ssm_oracle(few, rows, n(s)[i][ch])
        oracle.check(n(y[rows])[..., ch], want, err, "bf16", f"sequence {i}")
        oracle.check(n(h)[i][ch], hw, he, "f32", f"state {i}")


def test_selective_scan_with_the_callers_workspace():
    """A workspace of the caller's, full of NaN, used twice; one that is too small is replaced."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(18)
    kw = _ssm_inputs(r, "bf16", (1, 700), 96, 16, 1, True, True, True, True)
    want, hw = gdn.selective_scan(**kw)
    for size in (1 << 22, 16):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            y, h = gdn.selective_scan(**kw, workspace=ws)
            assert torch.equal(y, want) and torch.equal(h, hw)
    with pytest.raises(ValueError):
        gdn.selective_scan(**kw, workspace=torch.zeros(1 << 22, device="cuda"))


def test_selective_scan_slow_channels_over_a_long_document():
    """Steps so small that nothing decays over 70000 tokens: the sums of step sizes that carry states over chunks keep
    their precision (against 64 bits, a running sum of the same inputs)."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(19)
    T, D, N = 70001, 64, 4
    x, B = r.t(1, T, D), r.t(1, T, N)
    dt = r.t(1, T, D).abs() * 1e-6 + 1e-6
    A = -torch.rand(D, N, device="cuda") - 0.5
    y, h = gdn.selective_scan(x, dt, A, B, B, dt_softplus=False)
    # h_T = sum_t exp(A (S_T - S_t)) dt_t x_t B_t
    S = torch.cumsum(dt[0].double(), 0)
    want = torch.zeros(D, N, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    for k in range(N):
        term = torch.exp(A[:, k].double() * (S[-1] - S)) * (dt[0] .double() * x[0].double()) * B[0, :, k:k + 1].double()
        want[:, k], mag[:, k] = term.sum(0), term.abs().sum(0)
    # per token a decay and an update round (10 U), over what is left of each term
    bound = 10 * oracle.U * (T * mag) / 2
    assert ((h[0].double() - want).abs() <= bound).all()
    assert float((h[0].double() - want).norm() / want.norm()) < 1e-5


def test_selective_scan_slots_in_place():
    """States in a pool by index (one out of range: it starts from zero and leaves no state), advanced in place."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(9)
    D, N, lens = 24, 16, [40, 0, 129, 1500, 7]
    kw = _ssm_inputs(r, "bf16", (sum(lens) + 9,), D, N, 1, True, True, True, True)
    pool = r.t(8, D, N)
    before = pool.clone()
    idx = [3, 6, -1, 0, 8]
    out = torch.full((sum(lens) + 9, D), 3.0, dtype=torch.bfloat16, device="cuda")
    y, h = gdn.selective_scan(**kw, state_in=pool, state_out=pool, seq_offsets=offsets(lens), out=out,
                              state_index=torch.tensor(idx, dtype=torch.int32, device="cuda"))
    assert h is pool and (out[sum(lens):] == 3).all()
    at = np.concatenate([[0], np.cumsum(lens)])
    for i, slot in enumerate(idx):
        ok = 0 <= slot < 8
        rows = slice(at[i], at[i + 1])
        (want, err), (hw, he) = _ssm_oracle(kw, rows, n(before)[slot] if ok else np.zeros((D, N)))
        oracle.check(n(y)[rows], want, err, "bf16", f"sequence {i}")
        if ok:
            oracle.check(n(pool)[slot], hw, he, "f32", f"state {i}")
    rest = [1, 2, 4, 5, 7]
    assert torch.equal(pool[rest], before[rest])


def test_selective_scan_extreme_steps():
    """Step sizes from e^-30 to 60 and decay rates up to 400: decays from 1 to fully underflown; finite everywhere."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(10)
    kw = _ssm_inputs(r, "f32", (1, 1300), 8, 16, 1, True, True, False, True)
    kw["dt"] = torch.linspace(-30, 60, 1300, device="cuda")[None, :, None].expand(1, 1300, 8).contiguous()
    kw["A"] = -torch.logspace(-6, 2.6, 16, device="cuda").expand(8, 16).contiguous()
    kw["x"], kw["B"] = kw["x"] * 0.1, kw["B"] * 0.1
    s = r.t(1, 8, 16)
    y, h = gdn.selective_scan(**kw, state_in=s)
    (want, err), (hw, he) = _ssm_oracle(kw, 0, n(s)[0])
    oracle.check(n(y)[0], want, err, "f32", "out")
    oracle.check(n(h)[0], hw, he, "f32", "state")


def test_selective_scan_nan_stays_in_its_place():
    """A NaN input reaches its own channel from its token on, and nothing else: not earlier tokens, not other
    channels, not the other sequences of a packed batch."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(11)
    lens = [900, 700, 30]
    kw = _ssm_inputs(r, "f32", (sum(lens),), 16, 16, 1, False, True, True, True)
    ref, href = gdn.selective_scan(**kw, seq_offsets=offsets(lens))
    kw["x"] = kw["x"].clone()
    kw["x"][900 + 333, 5] = float("nan")
    y, h = gdn.selective_scan(**kw, seq_offsets=offsets(lens))
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[900 + 333: 1600, 5] = True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], ref[~bad])
    hb = torch.zeros_like(h, dtype=torch.bool)
    hb[1, 5] = True
    assert torch.isnan(h[hb]).all() and torch.equal(h[~hb], href[~hb])


@pytest.mark.parametrize("name", ["x", "dt"])
@pytest.mark.parametrize("T,N", [(1, 16), (9, 5), (70, 100), (1003, 16)])
def test_selective_scan_infinite_last_token(T, N, name):
    """An infinite input or step size in a sequence's last token makes that channel's state infinite with the sign
    of B (x > 0), not NaN, and changes no earlier output and no other channel."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(31)
    kw = _ssm_inputs(r, "f32", (2, T), 80, N, 1, True, True, True, True)
    kw["x"] = kw["x"].abs() + 0.5
    ref, href = gdn.selective_scan(**kw)
    kw[name] = kw[name].clone()
    kw[name][1, T - 1, 70] = float("inf")
    y, h = gdn.selective_scan(**kw)
    assert torch.equal(y[0], ref[0]) and torch.equal(h[0], href[0])
    assert torch.equal(y[1, :T - 1], ref[1, :T - 1])
    assert torch.equal(h[1, :70], href[1, :70]) and torch.equal(h[1, 71:], href[1, 71:])
    assert torch.equal(h[1, 70], kw["B"][1, T - 1, 0].float() * float("inf"))


@pytest.mark.parametrize("T", [1, 9, 70, 1003])
def test_selective_scan_infinite_rate(T):
    """A rate of minus infinity forgets everything at every token: that entry's state is the last token's own input
    dt' x B.  Bound: softplus (polynomial, exponential, reciprocal and four roundings) and two products, under 16
    half steps of fp32."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(32)
    kw = _ssm_inputs(r, "f32", (1, T), 80, 16, 1, False, False, False, True)
    kw["A"][70, 3] = float("-inf")
    y, h = gdn.selective_scan(**kw)
    dt, x, B = (kw[k][0, T - 1].double() for k in ("dt", "x", "B"))
    want = torch.log1p(torch.exp(dt[70])) * x[70] * B[0, 3]
    assert abs(float(h[0, 70, 3]) - float(want)) <= 16 * 2.0 ** -24 * abs(float(want))
    assert torch.isfinite(y).all() and torch.isfinite(h).all()


def test_selective_scan_stride_of_one_token():
    """With a single token its stride means nothing, however large."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(33)
    kw = _ssm_inputs(r, "f32", (2, 1), 20, 4, 1, True, True, True, True)
    ref = gdn.selective_scan(**kw)
    far = kw["x"].contiguous().as_strided((2, 1, 20), (20, 1 << 30, 1))
    got = gdn.selective_scan(**{**kw, "x": far})
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("kind,B,D,N,G,gate,skip,bias,softplus", [
    ("bf16", 128, 256, 16, 1, True, True, True, True), ("f32", 1, 1, 1, 1, False, False, False, False),
    ("bf16", 5, 96, 7, 3, True, False, True, True), ("f32", 3, 40, 256, 2, False, True, True, True),
    ("f32", 9, 64, 24, 1, True, True, True, True), ("bf16", 4, 24, 64, 1, True, True, False, True)])
def test_selective_step(kind, B, D, N, G, gate, skip, bias, softplus):
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(12)
    kw = _ssm_inputs(r, kind, (B,), D, N, G, gate, skip, bias, softplus)
    slots = B + 2
    pool = r.t(slots, D, N)
    before = pool.clone()
    idx = r.g.permutation(slots)[:B].astype(np.int32)
    if B > 2:
        idx[0], idx[2] = slots, -7
    out = torch.full((B, D), 5.0, dtype=kw["x"].dtype, device="cuda")
    y = gdn.selective_step(**kw, state=pool, state_index=torch.from_numpy(idx).cuda(), out=out)
    used = []
    for i, slot in enumerate(idx.tolist()):
        if not 0 <= slot < slots:
            assert (y[i] == 5).all()
            continue
        used.append(slot)
        (want, err), (hw, he) = _ssm_oracle(kw, slice(i, i + 1), n(before)[slot])
        oracle.check(n(y)[i: i + 1], want, err, kind, f"row {i}")
        oracle.check(n(pool)[slot], hw, he, "f32", f"state {i}")
    rest = [i for i in range(slots) if i not in used]
    assert torch.equal(pool[rest], before[rest])


# ---- rotary positions ----

ROTARY = [
    # kind, B, T, Hq, Hk, d, rot, interleaved, axes, position type
    ("bf16", 1, 1, 1, 1, 64, 64, False, 1, "int32"),
    ("bf16", 2, 37, 8, 2, 128, 64, False, 1, "int64"),
    ("bf16", 2, 37, 4, 4, 128, 128, True, 3, "int32"),
    ("f32", 1, 300, 3, 1, 96, 24, False, 1, None),
    ("f32", 3, 5, 2, 1, 80, 20, True, 2, "int64"),      # rot not a whole vector
    ("bf16", 1, 9, 2, 1, 7, 6, False, 1, "int64"),
    ("f32", 1, 11, 1, 1, 2, 2, True, 1, None),
    ("bf16", 1, 4, 300, 5, 256, 256, False, 4, "int32"),
    ("f32", 2, 700, 16, 16, 128, 32, True, 1, "int64"),
    ("bf16", 1, 50, 1, 1, 255, 254, False, 1, "int64"),
]


@pytest.mark.parametrize("kind,B,T,Hq,Hk,d,rot,interleaved,axes,ptype", ROTARY)
def test_rotary(kind, B, T, Hq, Hk, d, rot, interleaved, axes, ptype):
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(13 + d)
    rows = r.t(B, T, Hq + 2 * Hk, d, kind=kind)
    q, k = rows[:, :, :Hq], rows[:, :, Hq: Hq + Hk]
    f, scale = gdn.rotary_frequencies(rot, scaling="parts", factor=8.0)
    sections = None
    pairs = rot // 2
    if axes > 1:
        sections = [pairs - (axes - 1) * (pairs // axes)] + [pairs // axes] * (axes - 1)
    pos = None
    p = np.broadcast_to(np.arange(T) + 7, (1, B, T))
    if ptype:
        p = r.g.integers(-1000, 2 ** 24 if axes == 1 else 5000, (axes, B, T))
        pos = torch.from_numpy(p).to(getattr(torch, ptype)).cuda()
        pos = pos[0] if axes == 1 else pos
    fn = f.numpy()
    axis = np.repeat(np.arange(axes), sections or [pairs])
    theta = _angles(p, axis, fn)
    for inverse in (False, True):
        qo, ko = gdn.rotary(q, k, f.cuda(), pos, interleaved, sections, scale, inverse, position0=7)
        for got, x in ((qo, q), (ko, k)):
            want, err = oracle.rotary(n(x), theta, interleaved, np.float64(np.float32(scale)), inverse)
            oracle.check(n(got), want, err, kind)
    only, none = gdn.rotary(q, None, f.cuda(), pos, interleaved, sections, scale, False, position0=7)
    assert none is None
    first, _ = gdn.rotary(q, k, f.cuda(), pos, interleaved, sections, scale, False, position0=7)
    assert torch.equal(only, first)


def _angles(p, axis, f):
    """Angles reduced to one turn in extended precision (80 bits), so that the oracle's own are exact."""
    two_pi = np.longdouble("6.283185307179586476925286766559005768")
    theta = np.fmod(p[axis].astype(np.longdouble).transpose(1, 2, 0) * f.astype(np.longdouble), two_pi)
    return theta.astype(np.float64)


def test_rotary_in_place_and_heads_first():
    """In place on q and k inside one fused projection (v untouched), and on [B, H, T, d] memory, equal to the plain
    call bit for bit."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(14)
    f = gdn.rotary_frequencies(32)[0].cuda()
    for Hq, Hk in ((8, 2), (4, 4)):
        rows = r.t(2, 50, Hq + 2 * Hk, 64, kind="bf16")
        before = rows.clone()
        q, k = rows[:, :, :Hq], rows[:, :, Hq: Hq + Hk]
        qo, ko = gdn.rotary(q, k, f)
        gdn.rotary(q, k, f, q_out=q, k_out=k)
        assert torch.equal(q, qo) and torch.equal(k, ko)
        assert torch.equal(rows[:, :, Hq + Hk:], before[:, :, Hq + Hk:])
    hq, hk = r.t(2, 4, 50, 64).transpose(1, 2), r.t(2, 1, 50, 64).transpose(1, 2)
    qo, ko = gdn.rotary(hq, hk, f, interleaved=True)
    q2, k2 = torch.empty(2, 4, 50, 64, device="cuda").transpose(1, 2), torch.empty(2, 1, 50, 64, device="cuda").transpose(1, 2)
    gdn.rotary(hq, hk, f, interleaved=True, q_out=q2, k_out=k2)
    assert torch.equal(qo, q2) and torch.equal(ko, k2)


def test_rotary_inverse_is_the_gradient():
    """<J u, g> = <u, J^T g>: the inverse call is the transpose, against differences of the forward call."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(15)
    f = gdn.rotary_frequencies(64)[0].cuda()
    q, g, u = (r.t(1, 9, 2, 80) for _ in range(3))
    kw = dict(interleaved=True, scale=1.3)
    grad, _ = gdn.rotary(g, None, f, inverse=True, **kw)
    step = 0.25  # the call is linear: the difference is exact up to rounding
    plus, _ = gdn.rotary(q + step * u, None, f, **kw)
    minus, _ = gdn.rotary(q - step * u, None, f, **kw)
    lhs = float(((plus - minus).double() / (2 * step) * g.double()).sum())
    rhs = float((u.double() * grad.double()).sum())
    mag = float((u.double().abs() * grad.double().abs()).sum()) + float((plus.abs() * g.abs()).sum()) / step
    assert abs(lhs - rhs) <= 16 * oracle.U * 2 * mag


# ---- delta rule step ----

@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 12, 128, 128), (40, 16, 128, 128), (3, 1, 64, 128), (40, 13, 64, 64),
                                       (2, 5, 128, 64), (41, 13, 128, 64), (50, 11, 64, 128)])
@pytest.mark.parametrize("opts", [dict(), dict(erase=False), dict(exclusive=True), dict(epilogue=True)])
def test_delta_step(kind, B, H, dk, dv, opts):
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(16)
    opts = dict(opts)
    epilogue = opts.pop("epilogue", False)
    q, k, v = r.t(B, H, dk, kind=kind), r.t(B, H, dk, kind=kind, scale=3.0), r.t(B, H, dv, kind=kind)
    la, beta = -torch.nn.functional.softplus(r.t(B, H)), torch.sigmoid(r.t(B, H))
    gate, nw = (r.t(B, H, dv, kind=kind), r.t(dv)) if epilogue else (None, None)
    slots = B + 2
    pool = r.t(slots, H, dv, dk, scale=0.3)
    before = pool.clone()
    idx = r.g.permutation(slots)[:B].astype(np.int32)
    if B > 1:
        idx[1] = -1
        q[0, 0] = 0  # a zero query and key
        k[0, 0] = 0
    out = torch.full((B, H, dv), 5.0, device="cuda")
    o = gdn.delta_step(q, k, v, la, beta, pool, torch.from_numpy(idx).cuda(), gate=gate, norm_weight=nw, norm_eps=1e-5,
                       out=out, **opts)
    used = []
    for i, slot in enumerate(idx.tolist()):
        if slot < 0:
            assert (o[i] == 5).all()
            continue
        used.append(slot)
        (want, err), (sw, se) = oracle.delta_step(n(q)[i], n(k)[i], n(v)[i], n(la)[i], n(beta)[i], n(before)[slot],
                                                  gate=None if gate is None else n(gate)[i], weight=n(nw), eps=1e-5, **opts)
        oracle.check(n(o)[i], want, err, "f32", f"row {i}")
        oracle.check(n(pool)[slot], sw, se, "f32", f"state {i}")
    rest = [i for i in range(slots) if i not in used]
    assert torch.equal(pool[rest], before[rest])


def test_delta_step_equals_one_token_of_the_scan():
    """The step against ``forward`` on a single token (its chunk arithmetic in fp32), state and readout."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(17)
    B, H, d = 2, 3, 128
    q, k, v = r.t(B, 1, H, d), r.t(B, 1, H, d), r.t(B, 1, H, d)
    la, beta = -torch.nn.functional.softplus(r.t(1, B, 1, H)), torch.sigmoid(r.t(1, B, 1, H))
    s = r.t(1, B, H, d, d, scale=0.1)
    o, s2 = gdn.forward(q, k, v, la, beta, s)
    st = s[0].clone()
    o1 = gdn.delta_step(q[:, 0], k[:, 0], v[:, 0], la[0, :, 0], beta[0, :, 0], st)
    assert float((o1 - o[:, 0]).abs().max()) <= 1e-4 * float(o.square().mean().sqrt())
    assert float((st - s2[0]).abs().max()) <= 1e-4 * float(s2.square().mean().sqrt())
