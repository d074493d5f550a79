"""The seam's gradients as training hands them on and takes them, on the GPU."""
import pytest

from test_gpu_hybrid import SeamCase
from test_gpu_layer import Rng, _torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,lens,D", [("bf16", (2, 37), 96), ("f32", (5, 9), 33), ("bf16", (3000,), 64), ("f32", [5, 0, 31], 130)])
def test_gradients_whose_rows_are_not_contiguous(kind, lens, D):
    """An expanded value, a transposed buffer, every second channel: as their contiguous copies, also on another stream
    beside pending work of theirs."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    c = SeamCase(kind, lens, D, True, "sequence", True, True, 1.0, "plain")
    shape, dt = c.x.shape, c.x.dtype
    r = Rng(5)
    one = torch.ones((), dtype=dt, device="cuda").expand(shape)
    turned = r.t(*shape[:-2], D, shape[-2], kind=kind).transpose(-1, -2)
    second = r.t(*shape, 2, kind=kind)[..., 0]
    assert all(g.stride(-1) != 1 and g.shape == shape for g in (one, turned, second))
    for dh, dn in ((one, one), (turned, second), (second, one), (None, turned), (c.dh, one)):
        solid = [None if g is None else g.contiguous() for g in (dh, dn)]
        want = gdn.residual_norm_backward(*solid, c.x, c.y, **c.args())
        got = gdn.residual_norm_backward(dh, dn, c.x, c.y, **c.args())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(1_000_000)
        late = [torch.empty(c.x.numel(), dtype=dt, device="cuda").fill_(7) for _ in range(4)]  # blocks of the copies' size
        del late
        other = gdn.residual_norm_backward(dh, dn, c.x, c.y, **c.args(), stream=side)
        torch.cuda.synchronize()
        for a, b, o in zip(want, got, other):
            assert torch.equal(a, b) and torch.equal(a, o)


def test_gradients_that_do_not_fit_are_refused():
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    x = torch.zeros((2, 5, 8), device="cuda")
    for bad in (x[:1], x.bfloat16(), x.transpose(0, 1), x[..., :4], x.cpu()):
        with pytest.raises(ValueError):
            gdn.residual_norm_backward(bad, None, x, x)
        with pytest.raises(ValueError):
            gdn.residual_norm_backward(None, bad, x, x, weight=x[0, 0])
    turned = torch.zeros((2, 8, 5), device="cuda").transpose(1, 2)
    with pytest.raises(ValueError):  # a result's rows are contiguous
        gdn.residual_norm_backward(turned, None, x, x, dx=turned)


FORMS = [
    # kind, lens, D, y, gate, post, weight, alpha
    ("bf16", (2, 37), 96, True, "sequence", True, True, 1.0),
    ("f32", (3, 20), 130, True, "channel", False, True, 0.5),
    ("bf16", (65,), 64, True, None, True, False, 1.0),
    ("f32", [5, 0, 31], 33, True, "sequence", True, True, 1.0),
    ("bf16", (2, 9), 256, False, None, False, True, 1.0),
    ("f32", (2, 9), 256, False, None, False, True, 0.7),
    ("f32", (2, 9), 64, False, None, False, False, 0.7),
]


def _leaves(c):
    """The case's tensors as leaves: (arguments, those that are there)."""
    named = dict(x=c.x, y=c.y, gate=c.gate, post_weight=c.post, weight=c.weight)
    named = {k: None if t is None else t.detach().clone().requires_grad_() for k, t in named.items()}
    return dict(**named, residual_scale=c.alpha, eps=c.eps, seq_offsets=c.off), [t for t in named.values() if t is not None]


@pytest.mark.parametrize("kind,lens,D,has_y,gate,post,weight,alpha", FORMS)
def test_gradients_through_autograd(kind, lens, D, has_y, gate, post, weight, alpha):
    """The outputs and, with gradients of h, of n and of both, the gradients of the call by name, bit for bit."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    c = SeamCase(kind, lens, D, has_y, gate, post, weight, alpha, "plain")
    if not weight:
        c.dn = None
    eager = gdn.residual_norm(c.x, c.y, **c.args())
    moves = has_y or alpha != 1.0
    for use_h, use_n in ((True, True), (True, False), (False, True)):
        args, leaves = _leaves(c)
        h, nn = gdn.residual_norm(**args)
        assert torch.equal(h, eager[0]) and (h is args["x"]) == (not moves)
        assert (nn is None) == (not weight) and (nn is None or torch.equal(nn, eager[1]))
        use = [(t, g) for t, g, u in ((h, c.dh, use_h), (nn, c.dn, use_n)) if u and t is not None]
        if not use:
            continue
        got = torch.autograd.grad([t for t, _ in use], leaves, [g for _, g in use], allow_unused=True)
        named = c.args()
        if not use_n:
            named["weight"] = None
        if moves or use_n:
            want = gdn.residual_norm_backward(c.dh if use_h and moves else None, c.dn if use_n else None, c.x, c.y, **named)
            want = [w for w, t in zip(want, (c.x, c.y, c.gate, c.post, c.weight)) if t is not None]
        else:
            want = [None] * len(leaves)
        if use_h and not moves:  # h is x
            want[0] = c.dh if want[0] is None else want[0] + c.dh
        for g, w in zip(got, want):
            assert (g is None) == (w is None) and (w is None or torch.equal(g, w))


def test_training_step_through_autograd():
    """Two blocks, a loss by a sum (its gradient is one value, expanded), parameters that require gradients; against
    differences of the loss in 64 bits from the formulas.

    fp32 gradients are off by some 300 roundings of terms that may be tens of times their sum: 300 * 2^-24 * 50 = 9e-4 of
    their magnitudes.  The step to the fourth is 2e-10, 64 bits over the step 1e-13."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(6)
    B, T, D = 2, 11, 40
    x, W = r.t(B, T, D), r.t(D, D, scale=D ** -0.5)
    leaves = [r.t(B, D, scale=0.3, mean=0.4), r.t(D, scale=0.1, mean=1.0), r.t(D, scale=0.1, mean=1.0), r.t(D, scale=0.1, mean=1.0)]

    def end(h, n2):
        return (n2 * n2.sin()).sum() + h.sum()

    def loss(gate, post, w1, w2):
        h, n1 = gdn.residual_norm(x, weight=w1)
        assert h is x
        return end(*gdn.residual_norm(h, torch.tanh(n1 @ W), gate=gate, post_weight=post, weight=w2))

    def loss64(gate, post, w1, w2):
        norm = lambda z: z / ((z * z).mean(-1, keepdim=True) + 1e-6).sqrt()
        h = x.double() + gate[:, None] * post * norm(torch.tanh(w1 * norm(x.double()) @ W.double()))
        return end(h, w2 * norm(h))

    params = [t.clone().requires_grad_() for t in leaves]
    loss(*params).backward()
    step = 2.0 ** -8
    for i, (p, t) in enumerate(zip(params, leaves)):
        d = torch.randn(t.shape, generator=torch.Generator().manual_seed(i)).cuda().double()
        at = lambda s: float(loss64(*(u.double() + s * d if j == i else u.double() for j, u in enumerate(leaves))))
        slope = (8 * (at(step) - at(-step)) - (at(2 * step) - at(-2 * step))) / (12 * step)
        terms = p.grad.double() * d
        assert abs(slope - float(terms.sum())) <= 9e-4 * float(terms.abs().sum()), (i, slope, float(terms.sum()))


def test_what_does_not_go_with_gradients():
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    x, y = torch.randn(2, 5, 64, device="cuda"), torch.randn(2, 5, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda")
    for bad in (dict(out=x), dict(norm_out=torch.empty_like(x)), dict(stream=torch.cuda.Stream())):
        with pytest.raises(ValueError):
            gdn.residual_norm(x, y, weight=w, **bad)
    with torch.no_grad():
        want = gdn.residual_norm(x, y, weight=w)
        out = torch.empty_like(x)
        h, nn = gdn.residual_norm(x, y, weight=w, out=out, stream=torch.cuda.current_stream())
    assert h.data_ptr() == out.data_ptr() and not h.requires_grad and torch.equal(h, want[0]) and torch.equal(nn, want[1])
    h, nn = gdn.residual_norm(x, y, weight=w)
    assert h.requires_grad and nn.requires_grad
    (g,) = torch.autograd.grad(h.sum(), y, create_graph=True)
    with pytest.raises(RuntimeError):  # no second derivatives
        g.sum().backward()
    # values kept for the backward pass that a call writes over
    h, nn = gdn.residual_norm(x, y, weight=w)
    with torch.no_grad():
        gdn.residual_norm(x, y, weight=w, out=x)
    with pytest.raises(RuntimeError):
        nn.sum().backward()


@pytest.mark.parametrize("scale", [1.0, 1.0 + 1e-10, 1])
def test_a_scale_of_one_in_32_bits(scale):
    """Without y the residual stream then stays what it is, with gradients and without."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    x, w = torch.randn(3, 64, device="cuda", requires_grad=True), torch.ones(64, device="cuda")
    h, nn = gdn.residual_norm(x, weight=w, residual_scale=scale)
    with torch.no_grad():
        want = gdn.residual_norm(x, weight=w, residual_scale=scale)
    assert h is x and want[0] is x and torch.equal(nn, want[1]) and nn.requires_grad


def test_compiled_training_step():
    """The op's autograd formula, eagerly and traced."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    gdn.register_torch_ops()
    c = SeamCase("bf16", (2, 37), 96, True, "sequence", True, True, 0.9, "plain")
    want = gdn.residual_norm_backward(c.dh, c.dn, c.x, c.y, **c.args())

    def fn(x, y, gate, post, weight):
        h, nn = torch.ops.gdn.residual_norm(x, y, gate, post, weight, 0.9, 1e-6, None)
        return (h * c.dh).sum() + (nn * c.dn).sum()

    for f in (fn, torch.compile(fn, backend="aot_eager", fullgraph=True)):
        args, leaves = _leaves(c)
        f(*leaves).backward()
        for t, w in zip(leaves, want):
            assert torch.equal(t.grad, w)
    args, leaves = _leaves(c)
    torch.ops.gdn.residual_norm(leaves[0], leaves[1], None, None, leaves[4], 1.0, 1e-6, None)[1].sum().backward()
    assert leaves[0].grad is not None and leaves[4].grad is not None and leaves[2].grad is None


def test_captured_training_step():
    """Forward and gradients in one graph, replayed on new inputs with eager work between; the leaves are the graph's own
    and no eager graph of them is alive."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    c = SeamCase("bf16", (2, 150), 136, True, "sequence", True, True, 0.9, "plain")

    def step(x, y, gate, post, weight):
        h, nn = gdn.residual_norm(x, y, gate, post, weight, 0.9)
        loss = (h * c.dh).sum(-1) + nn.sum(-1)  # (n's gradient is expanded)
        return h, nn, *torch.autograd.grad(loss, (x, y, gate, post, weight), torch.ones_like(loss))

    def fresh():
        return [t.detach().clone().requires_grad_() for t in (c.x, c.y, c.gate, c.post, c.weight)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*fresh())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    leaves = fresh()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(*leaves)
    r = Rng(8)
    for i in range(3):
        new = [r.t(*t.shape).to(t.dtype) for t in leaves]
        with torch.no_grad():
            for t, v in zip(leaves, new):
                t.copy_(v)
        want = [t.detach().clone() for t in step(*(v.requires_grad_() for v in new))]
        torch.randn(1000, 1000, device="cuda").sum()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), f"replay {i}"
