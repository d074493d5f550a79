"""Infinite inputs and states of the selective scan: where the formula gives an infinity, the operators give it, at any
number of state entries and however a sequence is split."""
import pytest

from test_gpu_layer import Rng, offsets

pytestmark = pytest.mark.gpu

INF = float("inf")
ENTRIES = [1, 3, 5, 8, 12, 16, 20, 24, 33, 37, 64, 100, 256]


def _inputs(lead, D, N, kind="f32", seed=51, rate=1.0):
    """Positive inputs, B, C, skip and gate, so that every sum of the formula has one sign."""
    import torch

    r = Rng(seed)
    pos = lambda *s, k=kind: (r.t(*s, kind=k).abs() + 0.25).to(torch.bfloat16 if k == "bf16" else torch.float32)
    return dict(x=pos(*lead, D), dt=r.t(*lead, D, kind=kind, scale=0.5), A=-pos(D, N, k="f32") * rate, B=pos(*lead, N),
                C=pos(*lead, N), D=pos(D, k="f32"), z=pos(*lead, D))


@pytest.mark.parametrize("name", ["x", "dt"])
@pytest.mark.parametrize("T", [1, 9, 70, 1003])
@pytest.mark.parametrize("N", ENTRIES)
def test_last_token(N, T, name):
    """An infinite input or step size of the last token: output and state are infinite with the sign of C and of B,
    and nothing else changes."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    for sign in (1.0, -1.0):
        kw = _inputs((2, T), 80, N)
        kw["C"], kw["D"] = kw["C"] * sign, kw["D"] * sign
        ref, href = gdn.selective_scan(**kw)
        kw[name] = kw[name].clone()
        kw[name][1, T - 1, 70] = INF
        y, h = gdn.selective_scan(**kw)
        assert y[1, T - 1, 70] == sign * INF and (h[1, 70] == INF).all()
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[1, T - 1, 70] = True
        assert torch.equal(y[~hit], ref[~hit])
        h[1, 70] = href[1, 70]
        assert torch.equal(h, href)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 9, 70, 1003])
@pytest.mark.parametrize("N", [1, 5, 8, 16, 32, 64, 100])
def test_without_skip(N, T, kind, gate):
    """No D: an infinite last input reaches the output through the state alone."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    kw = _inputs((2, T), 80, N, kind)
    kw["D"], kw["z"] = None, kw["z"] if gate else None
    kw["x"][1, T - 1, 70] = INF
    for sign in (1.0, -1.0):
        y, h = gdn.selective_scan(**dict(kw, C=kw["C"] * sign))
        assert y[1, T - 1, 70] == sign * INF and (h[1, 70] == INF).all()
        assert not torch.isnan(y).any() and int(torch.isinf(y).sum()) == 1
    state = torch.zeros(2, 80, N, device="cuda")
    y = gdn.selective_step(**{k: t if k in ("A", "D") or t is None else t[:, T - 1].contiguous() for k, t in kw.items()}, state=state)
    assert y[1, 70] == INF and not torch.isnan(y).any() and int(torch.isinf(y).sum()) == 1


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T", [30, 70, 300])
@pytest.mark.parametrize("N", [1, 5, 12, 16, 20, 37, 64])
def test_stays_infinite(N, T, kind):
    """Behind an infinite input every output of the channel and its final state are infinite (decays above zero)."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    kw = _inputs((1, T), 70, N, kind, rate=0.3)
    ref, href = gdn.selective_scan(**kw)
    for at in (0, T // 2):
        new = dict(kw, x=kw["x"].clone())
        new["x"][0, at, 65] = INF
        y, h = gdn.selective_scan(**new)
        assert (y[0, at:, 65] == INF).all() and (h[0, 65] == INF).all()
        y[0, at:, 65], h[0, 65] = ref[0, at:, 65], href[0, 65]
        assert torch.equal(y, ref) and torch.equal(h, href)


@pytest.mark.parametrize("N", ENTRIES)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_step(N, kind):
    """The single-token step: an infinite input, step size or state entry."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    kw = _inputs((3,), 37, N, kind)
    state = torch.rand(3, 37, N, device="cuda")
    s0 = state.clone()
    ref = gdn.selective_step(**kw, state=s0)
    for name in ("x", "dt", "first", "last"):
        new, s = dict(kw), state.clone()
        if name in kw:
            new[name] = kw[name].clone()
            new[name][1, 20] = INF
        else:
            s[1, 20, 0 if name == "first" else N - 1] = INF
        y = gdn.selective_step(**new, state=s)
        assert y[1, 20] == INF, name
        if name in kw:
            assert (s[1, 20] == INF).all(), name
        else:
            assert int((s[1, 20] == INF).sum()) == 1, name
        assert not torch.isnan(y).any() and not torch.isnan(s).any()
        y[1, 20], s[1, 20] = ref[1, 20], s0[1, 20]
        assert torch.equal(y, ref) and torch.equal(s, s0)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [(1, 300), (1, 1003), (1, 5000), (3, 700), [40, 1003, 0, 5000, 300]])
@pytest.mark.parametrize("N", [1, 5, 16, 37, 64])
def test_decays_whose_product_rounds_to_zero(N, lens, kind):
    """A sequence is split into chunks that each forget all of a finite state (e^-1 to e^-50 a token): an infinite one,
    carried in or from an input, stays."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    packed = isinstance(lens, list)
    kw = _inputs((sum(lens),) if packed else lens, 70, N, kind, rate=5.0)
    B, longest = (len(lens), 3) if packed else (lens[0], 0)
    first, last = (sum(lens[:3]), sum(lens[:4])) if packed else (0, lens[1])  # rows of sequence `longest`
    off = offsets(lens) if packed else None
    state = torch.rand(B, 70, N, device="cuda")
    ref, href = gdn.selective_scan(**kw, state_in=state, seq_offsets=off)
    assert torch.isfinite(ref).all() and torch.isfinite(href).all()
    rows = lambda y: y if packed else y[longest]
    for at in (None, 0, (last - first) // 2, last - first - 40):
        new, s = dict(kw), state.clone()
        if at is None:
            s[longest, 65], at = INF, 0
        else:
            new["x"] = kw["x"].clone()
            rows(new["x"])[first + at, 65] = INF
        y, h = gdn.selective_scan(**new, state_in=s, seq_offsets=off)
        assert (rows(y)[first + at: last, 65] == INF).all() and (h[longest, 65] == INF).all()
        rows(y)[first + at: last, 65], h[longest, 65] = rows(ref)[first + at: last, 65], href[longest, 65]
        assert torch.equal(y, ref) and torch.equal(h, href)


@pytest.mark.parametrize("T", [20, 300, 1003, 5000])
def test_rate_and_state_infinite(T):
    """A rate of minus infinity forgets at once: exp(-inf) * inf is no number, however the sequence is split."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    kw = _inputs((1, T), 70, 16)
    ref, href = gdn.selective_scan(**kw)
    new = dict(kw, A=kw["A"].clone(), x=kw["x"].clone())
    new["A"][65, 3], new["x"][0, 2, 65] = -INF, INF
    y, h = gdn.selective_scan(**new)
    assert torch.isnan(h[0, 65, 3]) and torch.isnan(y[0, 3:, 65]).all() and y[0, 2, 65] == INF
    assert (h[0, 65, torch.arange(16) != 3] == INF).all()
    y[0, :, 65], h[0, 65] = ref[0, :, 65], href[0, 65]
    assert torch.equal(y, ref) and torch.equal(h, href)
