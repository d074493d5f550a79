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
