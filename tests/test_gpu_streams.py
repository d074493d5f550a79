"""Calls on a stream that is not the current one: what a call allocates shares no memory with work that is still
pending on the current stream, and what it returns may be used and freed there."""
import pytest

from test_gpu_layer import Rng, _ssm_inputs

pytestmark = pytest.mark.gpu

LONG = 20_000_000  # cycles of waiting on the device, some ten milliseconds


def _calls():
    """name -> (call(stream), sizes in bytes of what it allocates)."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    r = Rng(61)
    B, T, D, N, H, d = 3, 1200, 136, 16, 4, 64
    w, x, t = r.t(D, 4), r.t(B, T, D), r.t(B, D)
    kw, tk = _ssm_inputs(r, "f32", (B, T), D, N, 1, True, True, True, True), _ssm_inputs(r, "f32", (B,), D, N, 1, True, True, True, True)
    q, f = r.t(B, T, H, d), gdn.rotary_frequencies(d)[0].cuda()
    q0 = q[:, 0].contiguous()
    la, beta = -r.t(B, H).abs(), torch.sigmoid(r.t(B, H))
    cs, hs, S = r.t(B, 3, D), r.t(B, D, N), r.t(B, H, d, d)
    p = gdn.gdn_ssm_problem_t(B=B, T=T, D=D, N=N, G=1, dtype=gdn.GDN_DTYPE_F32)
    ws = gdn.gdn_ssm_workspace_bytes(p)
    assert ws
    many = lambda y: y if isinstance(y, tuple) else (y,)
    out = {
        "conv": (lambda s: gdn.causal_conv(x, w, stream=s), [x.numel() * 4, cs.numel() * 4]),
        "conv step": (lambda s: gdn.causal_conv_step(t, w, None, cs.clone() if s is None else cs, stream=s), [t.numel() * 4]),
        "scan": (lambda s: gdn.selective_scan(**kw, stream=s), [x.numel() * 4, hs.numel() * 4, ws]),
        "step": (lambda s: gdn.selective_step(**tk, state=hs.clone() if s is None else hs, stream=s), [t.numel() * 4]),
        "rotary": (lambda s: gdn.rotary(q, q, f, stream=s), [q.numel() * 4]),
        "delta step": (lambda s: gdn.delta_step(q0, q0, q0, la, beta, S.clone() if s is None else S, stream=s), [q0.numel() * 4]),
    }
    # the scans themselves, the epilogue's weight a view that the call copies
    sq, sv = r.t(1, 700, H, d), r.t(1, 700, H, d)
    gate, nw = r.t(1, 700, H, d), r.t(d, 2)[:, 0]
    sla, sbeta = -r.t(1, 1, 700, H).abs(), torch.sigmoid(r.t(1, 1, 700, H))
    fla = -r.t(1, 1, 7, H).abs()
    kw2 = dict(gate=gate, norm_weight=nw)
    ws = gdn.workspace_bytes(1, 700, H, d, d, "f32")
    assert ws
    p = gdn.gdn_vda_problem_t(B=1, T=700, H=H, dk=d, dv=d, frame=100, dtype=gdn.GDN_DTYPE_F32)
    fws = gdn.gdn_vda_workspace_bytes(p, gdn.DIRECTIONS["fwd"])
    sizes = [sq.numel() * 4, H * d * d * 4, d * 4]
    out["token scan"] = (lambda s: gdn.forward(sq, sq, sv, sla, sbeta, stream=s, **kw2), sizes + [ws])
    out["frame-wise scan"] = (lambda s: gdn.vda_forward(sq, sq, sv, fla, sbeta, frame=100, stream=s, **kw2), sizes + [max(fws, 1)])
    return {k: ((lambda s, fn=fn: many(fn(s))), sizes) for k, (fn, sizes) in out.items()}


NAMES = ["conv", "conv step", "scan", "step", "rotary", "delta step", "token scan", "frame-wise scan"]


@pytest.mark.parametrize("name", NAMES)
def test_results_share_no_memory_with_pending_work(name):
    """Blocks of the very sizes that the call allocates are freed on the current stream while a fill of them is still
    to come there."""
    import torch

    call, sizes = _calls()[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(LONG)
    late = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in sizes for _ in range(3)]
    taken = {t.data_ptr() for t in late}
    del late
    got = call(side)
    assert not taken & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_results_freed_on_the_current_stream(name):
    """A result that the current stream has still to read is freed: the side stream's next tensors leave it alone."""
    import torch

    call, _ = _calls()[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(LONG)
    copies = [t.clone() for t in got]
    shapes = [t.shape for t in got]
    del got
    with torch.cuda.stream(side):
        junk = [torch.full(s, float("nan"), device="cuda") for s in shapes for _ in range(3)]
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)
    del junk


@pytest.mark.parametrize("name", ["conv step", "step", "delta step"])
def test_given_outputs_and_states(name):
    """Steps into outputs and states made before the side stream waits: rows with a slot are written, the others keep
    what the current stream put there, and states advance as on the current stream."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    r = Rng(62)
    B, D, N, H, d = 5, 136, 16, 4, 64
    index = torch.tensor([3, -1, 0, 5, 1], dtype=torch.int32, device="cuda")
    w, x, q = r.t(D, 4), r.t(B, D), r.t(B, H, d)
    kw = _ssm_inputs(r, "f32", (B,), D, N, 1, True, True, True, True)
    la, beta = -r.t(B, H).abs(), torch.sigmoid(r.t(B, H))
    pool = {"conv step": r.t(5, 3, D), "step": r.t(5, D, N), "delta step": r.t(5, H, d, d)}[name]
    call = {"conv step": lambda s, o, **k: gdn.causal_conv_step(x, w, None, s, state_index=index, out=o, **k),
            "step": lambda s, o, **k: gdn.selective_step(**kw, state=s, state_index=index, out=o, **k),
            "delta step": lambda s, o, **k: gdn.delta_step(q, q, q, la, beta, s, index, out=o, **k)}[name]
    like = q if name == "delta step" else x
    want, wanted = torch.full_like(like, 3.0), pool.clone()
    call(wanted, want)
    assert (want[[1, 3]] == 3).all() and not (want[[0, 2, 4]] == 3).any()
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda._sleep(LONG)
        out, state = torch.full_like(like, 3.0), pool.clone()
        side.wait_stream(torch.cuda.current_stream())
        assert call(state, out, stream=side).data_ptr() == out.data_ptr()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want) and torch.equal(state, wanted)
