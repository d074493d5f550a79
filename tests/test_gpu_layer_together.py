"""The layer operators as they run together, and in a program's surroundings:
prompt and single tokens through convolution, rotary positions and the delta
scan or the selective scan; graph capture and replay; another stream; guarded
and poisoned buffers; offsets beyond 32 bits; torch.compile."""
import numpy as np
import pytest

import layer_oracle as oracle
from test_gpu_layer import Rng, _ssm_inputs, n, offsets

pytestmark = pytest.mark.gpu


class DeltaLayer:
    """x -> convolution of the q, k and v channels -> rotary q, k -> delta scan with the readout epilogue."""

    def __init__(self, r, H, d):
        import gated_delta_rule_scan_amd as gdn

        self.H, self.d = H, d
        self.w = r.t(3 * H * d, 4, scale=0.5)
        self.freq = gdn.rotary_frequencies(d // 2)[0].cuda()
        self.nw = r.t(d, mean=1.0, scale=0.1)

    def prompt(self, x, la, beta, gate):
        import gated_delta_rule_scan_amd as gdn

        B, T, H, d = x.shape[0], x.shape[1], self.H, self.d
        u, conv = gdn.causal_conv(x, self.w)
        q, k, v = (u[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3))
        q, k = gdn.rotary(q, k, self.freq)
        o, S = gdn.forward(q, k, v.contiguous(), la[None], beta[None], None, gate=gate, norm_weight=self.nw)
        return o, conv, S[0]

    def token(self, x, la, beta, gate, conv, S, index, at):
        import gated_delta_rule_scan_amd as gdn

        H, d = self.H, self.d
        u = gdn.causal_conv_step(x, self.w, None, conv, state_index=index)
        q, k, v = (u[:, i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3))
        q, k = gdn.rotary(q[:, None], k[:, None], self.freq, at[:, None])
        return gdn.delta_step(q[:, 0], k[:, 0], v.contiguous(), la, beta, S, index, gate=gate, norm_weight=self.nw)


def test_delta_layer_prompt_then_tokens():
    """A prompt and then single tokens, states in a pool, equals the longer prompt (the scan's fp32 chunk arithmetic
    against the step's: the framework's fp32 tolerance)."""
    import torch

    r = Rng(21)
    B, T, more, H, d = 2, 137, 5, 3, 64
    L = DeltaLayer(r, H, d)
    x, gate = r.t(B, T + more, 3 * H * d), r.t(B, T + more, H, d)
    la = -torch.nn.functional.softplus(r.t(B, T + more, H) - 3.0)
    beta = torch.sigmoid(r.t(B, T + more, H))
    want, cw, Sw = L.prompt(x, la, beta, gate)
    cut = lambda t: t[:, :T].contiguous()
    o, conv, S = L.prompt(cut(x), cut(la), cut(beta), cut(gate))
    index = torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    cpool, spool = r.t(6, 3, 3 * H * d), r.t(6, H, d, d)
    cpool[index.long()], spool[index.long()] = conv, S
    outs = [o]
    for i in range(T, T + more):
        at = torch.full((B,), i, dtype=torch.int64, device="cuda")
        one = lambda t: t[:, i].contiguous()
        outs.append(L.token(one(x), one(la), one(beta), one(gate), cpool, spool, index, at)[:, None])
    got = torch.cat(outs, 1)
    rms = lambda t: float(t.square().mean().sqrt())
    assert float((got - want).abs().max()) <= 1e-4 * rms(want)
    assert torch.equal(cpool[index.long()], cw)
    assert float((spool[index.long()] - Sw).abs().max()) <= 1e-4 * rms(Sw)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_ssm_layer_prompt_pieces_and_tokens(kind):
    """Convolution and selective scan: a packed batch in one call, in two pieces with the states carried, and token by
    token, all against the oracle of the whole sequences."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    r = Rng(22)
    D, N, lens = 24, 16, [150, 1, 1100]
    rows = sum(lens)
    w, cb = r.t(D, 4, scale=0.5), r.t(D)
    kw = _ssm_inputs(r, kind, (rows,), D, N, 1, True, True, True, True)
    x = kw.pop("x")
    at = np.concatenate([[0], np.cumsum(lens)])
    u, conv = gdn.causal_conv(x, w, cb, seq_offsets=offsets(lens))
    y, h = gdn.selective_scan(u, **kw, seq_offsets=offsets(lens))
    for i in range(3):
        s = slice(at[i], at[i + 1])
        take = lambda t: n(t)[s]
        (want, err), (hw, he) = oracle.ssm(take(u), take(kw["dt"]), n(kw["A"]), take(kw["B"]), take(kw["C"]), n(kw["D"]),
                                           take(kw["z"]), n(kw["dt_bias"]), True, np.zeros((D, N)))
        oracle.check(n(y)[s], want, err, kind)
        oracle.check(n(h)[i], hw, he, "f32")
        # the last sequence again: a piece, then tokens, with the states carried in place
        if i == 2:
            cut, end = at[2] + 1090, at[3]
            c2, h2 = torch.zeros(1, 3, D, dtype=x.dtype, device="cuda"), torch.zeros(1, D, N, device="cuda")
            part = lambda t: t[at[2]:cut]
            up, _ = gdn.causal_conv(part(x)[None], w, cb, c2, state_out=c2)
            assert torch.equal(up[0], u[at[2]:cut])
            rest = {k: v for k, v in kw.items() if k not in ("dt", "B", "C", "z")}
            gdn.selective_scan(up, **{k: part(kw[k])[None] for k in ("dt", "B", "C", "z")}, **rest, state_in=h2, state_out=h2)
            for t in range(cut, end):
                ut = gdn.causal_conv_step(x[t:t + 1], w, cb, c2)
                assert torch.equal(ut[0], u[t])
                yt = gdn.selective_step(ut, **{k: kw[k][t:t + 1] for k in ("dt", "B", "C", "z")}, **rest, state=h2)
                j = t - at[2]
                oracle.check(n(yt), want[j:j + 1], 2 * err[j:j + 1], kind)
            oracle.check(n(h2)[0], hw, 2 * he, "f32")
            assert torch.equal(c2[0], conv[2])


def _all_calls(r, kind="bf16"):
    """name -> (function of fresh static inputs, those inputs); every entry point once, outputs and states returned."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    B, T, D, N, H, d = 3, 1200, 136, 16, 4, 64
    lens = [700, 0, 500]
    off = offsets(lens)
    idx = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    w = r.t(D, 4)
    cx, cs = r.t(B, T, D, kind=kind), r.t(4, 3, D, kind=kind)
    px = r.t(T, D, kind=kind)
    sk = _ssm_inputs(r, kind, (T,), D, N, 1, True, True, True, True)
    dk = _ssm_inputs(r, kind, (B, T), D, N, 2, False, True, True, True)
    tk = _ssm_inputs(r, kind, (B,), D, N, 1, True, True, True, True)
    hs = r.t(4, D, N)
    q, k = r.t(B, 60, H, d, kind=kind), r.t(B, 60, 2, d, kind=kind)
    f = gdn.rotary_frequencies(d)[0].cuda()
    sq, skk, sv = (r.t(B, H, d, kind=kind) for _ in range(3))
    la, beta, S = -r.t(B, H).abs(), torch.sigmoid(r.t(B, H)), r.t(4, H, d, d)
    tx = r.t(B, D, kind=kind)

    def conv(x, s, **kw):
        return gdn.causal_conv(x, w, None, s, state_index=idx, state_out=s, **kw) if x.dim() == 3 else \
            gdn.causal_conv(x, w, seq_offsets=off, **kw)

    return {
        "conv": (lambda x, s, **o: conv(x, s, **o), dict(x=cx, s=cs)),
        "conv packed": (lambda x, **o: conv(x, None, **o), dict(x=px)),
        "conv step": (lambda x, s, **o: (gdn.causal_conv_step(x, w, None, s, state_index=idx, out=torch.zeros_like(x), **o), s),
                      dict(x=tx, s=cs.clone())),
        "ssm packed": (lambda **k: gdn.selective_scan(seq_offsets=off, **k), sk),
        "ssm": (lambda **k: gdn.selective_scan(**k), dk),
        "ssm step": (lambda s, **k: (gdn.selective_step(state=s, state_index=idx, out=torch.zeros(B, D, dtype=tx.dtype, device="cuda"), **k), s),
                     dict(tk, s=hs)),
        "rotary": (lambda q, k, **o: gdn.rotary(q, k, f, **o), dict(q=q, k=k)),
        "delta step": (lambda q, k, v, s, **o: (gdn.delta_step(q, k, v, la, beta, s, idx, out=torch.zeros(B, H, d, device="cuda"), **o), s),
                       dict(q=sq, k=skk, v=sv, s=S)),
    }


NAMES = ["conv", "conv packed", "conv step", "ssm packed", "ssm", "ssm step", "rotary", "delta step"]


def _clone(kw):
    import torch

    return {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in kw.items()}


@pytest.mark.parametrize("name", NAMES)
def test_capture_and_replay(name):
    """Captured once, replayed three times on new inputs with eager work between: every replay equals an eager call bit
    for bit (in-place states included)."""
    import torch

    r = Rng(23)
    fn, kw = _all_calls(r)[name]
    vary = [k for k in ("x", "q", "v", "s") if k in kw]
    start = _clone(kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn(**_clone(kw))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = fn(**kw)
    for i in range(3):
        new = {k: r.t(*start[k].shape).to(start[k].dtype) for k in vary}
        for k in vary:
            kw[k].copy_(new[k])
        want = fn(**{**_clone(kw), **{k: v.clone() for k, v in new.items()}})
        want = [w.clone() for w in want]
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b) or (name == "conv" and torch.equal(a[[0, 2]], b[[0, 2]])), f"replay {i}"


@pytest.mark.parametrize("name", NAMES)
def test_repeats_and_other_streams_are_bitwise_equal(name):
    """Twice the same, and on a stream that is not the current one while the current stream allocates and writes."""
    import torch

    fn, kw = _all_calls(Rng(24))[name]
    first = [t.clone() for t in fn(**_clone(kw))]
    for a, b in zip(first, fn(**_clone(kw))):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    for _ in range(3):
        own = _clone(kw)
        side.wait_stream(torch.cuda.current_stream())
        got = fn(**own, stream=side)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(first, got):
            assert torch.equal(a, b)
        del junk, got, own


G = 4096


def _guarded(t):
    import torch

    size = t.numel() * t.element_size()
    whole = torch.full((size + 2 * G,), 0x5A, dtype=torch.uint8, device="cuda")
    view = whole[G:G + size].view(t.dtype).view(t.shape)
    view.copy_(t)
    return view, whole


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("name", NAMES)
def test_guard_zones_and_poisoned_outputs(name, kind):
    """Every buffer sits between guard zones that stay intact; inputs keep their values; poisoned outputs are written
    everywhere (an equal call on other buffers gives the same bits)."""
    import torch

    fn, kw = _all_calls(Rng(25), kind)[name]
    want = [t.clone() for t in fn(**_clone(kw))]
    wholes, own = [], {}
    for k, v in kw.items():
        if isinstance(v, torch.Tensor):
            v, whole = _guarded(v)
            wholes.append(whole)
        own[k] = v
    if "step" not in name:
        outs = []
        for k in (("q_out", "k_out") if name == "rotary" else ("out",)):
            out, whole = _guarded(torch.full_like(want[len(outs)], float("nan")))
            wholes.append(whole)
            own[k] = out
            outs.append(out)
    got = fn(**own)
    torch.cuda.synchronize()
    for whole in wholes:
        assert (whole[:G] == 0x5A).all() and (whole[-G:] == 0x5A).all()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for k, v in kw.items():
        if isinstance(v, torch.Tensor) and k != "s":
            assert torch.equal(own[k], v), k


def test_offsets_beyond_32_bits():
    """Rows more than 2^32 bytes apart: two sequences at the ends of one 9 GB buffer, states in far slots."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    r = Rng(26)
    T, D, N = 70, 64, 16
    buf = torch.zeros((1 << 32) + (1 << 29), dtype=torch.bfloat16, device="cuda")
    far = 1 << 32  # elements
    view = lambda at, t: torch.as_strided(buf, (2, t, D), (far, D, 1), at)
    x, out, dt = view(0, T), view(1 << 20, T), view(1 << 21, T)
    small, sdt = r.t(2, T, D, kind="bf16"), r.t(2, T, D, kind="bf16", scale=0.5)
    x.copy_(small)
    dt.copy_(sdt)
    w = r.t(D, 4)
    want, _ = gdn.causal_conv(small, w)
    gdn.causal_conv(x, w, out=out)
    assert torch.equal(out, want)
    A, B = -torch.exp(r.t(D, N)), r.t(2, T, N, kind="bf16")
    want, hw = gdn.selective_scan(small, sdt, A, B, B)
    got, h = gdn.selective_scan(x, dt, A, B, B, out=out)
    assert torch.equal(got, want) and torch.equal(h, hw)
    f = gdn.rotary_frequencies(32)[0].cuda()
    want, _ = gdn.rotary(small[:, :, None], None, f)
    got, _ = gdn.rotary(x[:, :, None], None, f, q_out=out[:, :, None])
    assert torch.equal(got, want)
    # packed rows far apart: token stride of 2^26 elements, 70 rows
    px, po = (torch.as_strided(buf, (64, D), (1 << 26, 1), at) for at in (1 << 10, 1 << 11))
    px.copy_(small[0, :64])
    want, _ = gdn.causal_conv(small[0, :64].contiguous(), w, seq_offsets=offsets([30, 34]))
    gdn.causal_conv(px, w, seq_offsets=offsets([30, 34]), out=po)
    assert torch.equal(po, want)
    del buf, x, out, dt, px, po
    # a delta state pool of 2^32 elements and more
    H, d = 4, 128
    slots = (1 << 32) // (H * d * d) + 2
    pool = torch.zeros((slots, H, d, d), device="cuda")
    q, k, v = (r.t(1, H, d) for _ in range(3))
    la, beta = -r.t(1, H).abs(), torch.sigmoid(r.t(1, H))
    one = r.t(1, H, d, d)
    pool[slots - 1] = one[0]
    o = gdn.delta_step(q, k, v, la, beta, pool, torch.tensor([slots - 1], dtype=torch.int32, device="cuda"))
    o1 = gdn.delta_step(q, k, v, la, beta, one)
    assert torch.equal(o, o1) and torch.equal(pool[slots - 1], one[0])


def test_compiled_calls_equal_eager():
    import torch

    import gated_delta_rule_scan_amd as gdn

    gdn.register_torch_ops()
    r = Rng(27)
    B, T, D, N, H, d = 2, 90, 64, 16, 2, 64
    w, x = r.t(D, 4), r.t(B, T, D, kind="bf16")
    kw = _ssm_inputs(r, "bf16", (B, T), D, N, 1, True, True, True, True)
    q, f = r.t(B, T, H, d), gdn.rotary_frequencies(d)[0].cuda()
    la, beta, S = -r.t(B, H).abs(), torch.sigmoid(r.t(B, H)), r.t(B, H, d, d)

    def fn(x, q, S):
        u, c = torch.ops.gdn.causal_conv(x, w, None, None, "silu", None)
        y, h = torch.ops.gdn.selective_scan(u, kw["dt"], kw["A"], kw["B"], kw["C"], kw["D"], kw["z"], kw["dt_bias"], True,
                                            None, None)
        a, b = torch.ops.gdn.rotary(q, q, f, None, False, None, 1.0, False, 0)
        o = torch.ops.gdn.delta_step(a[:, 0].contiguous(), b[:, 1].contiguous(), q[:, 2].contiguous(), la, beta, S, None,
                                     True, False, None, None, 1e-6)
        return y, h, c, o + 1.0, S * 2.0

    S1, S2 = S.clone(), S.clone()
    got = torch.compile(fn, backend="aot_eager", fullgraph=True)(x, q, S1)
    want = fn(x, q, S2)
    for a, b in zip(got + (S1,), want + (S2,)):
        assert torch.equal(a, b)


def test_binding_refusals():
    """What the binding refuses before any launch: shapes, types, devices, missing states, memory that would meet."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    r = Rng(28)
    x, w, D, N = r.t(2, 9, 16), r.t(16, 4), 16, 8
    kw = _ssm_inputs(r, "f32", (2, 9), D, N, 2, True, True, True, True)
    kw.pop("x")
    i2 = torch.zeros(2, dtype=torch.int32, device="cuda")
    bad = [
        lambda: gdn.causal_conv(x[0], w), lambda: gdn.causal_conv(x, w[:8]), lambda: gdn.causal_conv(x, w.bfloat16()),
        lambda: gdn.causal_conv(x, w.t().contiguous().t()), lambda: gdn.causal_conv(x, w, activation="relu"),
        lambda: gdn.causal_conv(x.transpose(1, 2), r.t(9, 4)), lambda: gdn.causal_conv(x, w, bias=r.t(15)),
        lambda: gdn.causal_conv(x, w, state_in=r.t(3, 3, 16)), lambda: gdn.causal_conv(x, w, state_in=r.t(2, 2, 16)),
        lambda: gdn.causal_conv(x, w, state_in=r.t(2, 3, 16, kind="bf16")), lambda: gdn.causal_conv(x, w, state_index=i2),
        lambda: gdn.causal_conv(x, w, state_in=r.t(5, 3, 16), state_index=i2.long(), want_state=False),
        lambda: gdn.causal_conv(x, w, seq_offsets=i2), lambda: gdn.causal_conv(x[0], w, seq_offsets=i2.long()),
        lambda: gdn.causal_conv(x, w, out=x.bfloat16()), lambda: gdn.causal_conv(x, w.cpu()),
        lambda: gdn.causal_conv_step(x[:, 0], w), lambda: gdn.causal_conv_step(x, w, state=r.t(2, 3, 16)),
        lambda: gdn.causal_conv_step(x[:, 0], w, state=r.t(3, 3, 16)),
        lambda: gdn.selective_scan(x, **dict(kw, dt=kw["dt"][:, :8])), lambda: gdn.selective_scan(x, **dict(kw, A=kw["A"][:8])),
        lambda: gdn.selective_scan(x, **dict(kw, B=kw["B"].bfloat16())), lambda: gdn.selective_scan(x, **dict(kw, z=x[..., :8])),
        lambda: gdn.selective_scan(x, **dict(kw, C=kw["C"][..., :1, :])),
        lambda: gdn.selective_scan(x, **dict(kw, B=r.t(2, 9, 3, N), C=r.t(2, 9, 3, N))),
        lambda: gdn.selective_scan(x, **kw, state_in=r.t(2, D, N + 1)), lambda: gdn.selective_step(x, **kw, state=r.t(2, D, N)),
        lambda: gdn.rotary(x, None, torch.ones(2, dtype=torch.float64, device="cuda")),
        lambda: gdn.rotary(x[:, :, None], None, torch.ones(2, device="cuda")),
        lambda: gdn.rotary(x[:, :, None], None, torch.ones(2, dtype=torch.float64, device="cuda"), i2),
        lambda: gdn.rotary(x[:, :, None], x[:, :8, None], torch.ones(2, dtype=torch.float64, device="cuda")),
        lambda: gdn.rotary(x[:, :, None], None, torch.ones(2, dtype=torch.float64, device="cuda"),
                           torch.zeros(3, 2, 9, dtype=torch.int32, device="cuda")),
        lambda: gdn.delta_step(x, x, x, i2, i2, x), lambda: gdn.causal_conv(torch._neg_view(x), w),
        lambda: gdn.selective_scan(x, **dict(kw, z=torch._neg_view(kw["z"]))),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")
    for call in (lambda: gdn.causal_conv(x, w, out=x), lambda: gdn.selective_scan(x, **kw, out=x),
                 lambda: gdn.causal_conv(x, r.t(16, 5)),
                 lambda: gdn.rotary(x[:, :, None], None, torch.ones(9, dtype=torch.float64, device="cuda"))):
        with pytest.raises(gdn.GdnError):
            call()
