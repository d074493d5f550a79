"""Rows of an output that belong to no sequence: behind the last sequence of a packed batch, and a step's rows
without a slot.  An output that the call makes holds zeros there, whatever its memory held before; one that is given
keeps what it held."""
import numpy as np
import pytest

from test_gpu_layer import Rng, _ssm_inputs, offsets

pytestmark = pytest.mark.gpu


def _torch():
    import torch

    return torch


def _poison(shape, dtype):
    """Leave blocks full of NaN to the allocator, of the size that the next tensor of this shape takes."""
    torch = _torch()
    blocks = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(8)]
    del blocks


def _compare(call, like, used, shape=None, dtype=None):
    """``call(out)`` on a given output and on none: equal rows where ``used``, elsewhere the given ones and zeros; and
    what else the call returns (states) equal."""
    torch = _torch()
    shape, dtype = shape or like.shape, dtype or like.dtype
    given = torch.full(shape, 3.0, dtype=dtype, device="cuda")
    first = call(given)
    _poison(shape, dtype)
    second = call(None)
    y, z = first[0], second[0]
    assert y.data_ptr() == given.data_ptr() and z.shape == y.shape
    rest = torch.ones(shape[0], dtype=torch.bool, device="cuda")
    rest[used] = False
    assert torch.equal(z[used], y[used]) and not torch.isnan(y[used]).any()
    assert (y[rest] == 3).all() and (z[rest] == 0).all()
    for a, b in zip(first[1:], second[1:]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,lens,D", [(300, [100, 0, 57], 64), (300, [100, 0, 57], 33), (5000, [1, 1999], 72), (40, [0, 0], 8),
                                      (7, [3], 1), (70000, [20000, 0], 1032), (129, [129, 0], 24)])
def test_conv(kind, T, lens, D):
    import gated_delta_rule_scan_amd as gdn

    r = Rng(41)
    x, w, s = r.t(T, D, kind=kind), r.t(D, 4), r.t(len(lens), 3, D, kind=kind)
    _compare(lambda out: gdn.causal_conv(x, w, None, s, seq_offsets=offsets(lens), out=out), x, slice(0, sum(lens)))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,lens,D,N,G", [(30, [7, 5], 70, 16, 1), (700, [300, 0, 101], 72, 16, 2), (513, [40, 200], 66, 40, 1),
                                          (513, [0, 0], 66, 100, 1), (2000, [1], 300, 8, 3), (1000, [999], 5, 3, 1),
                                          (1000, [990, 10], 130, 16, 1), (3, [2, 0], 8, 256, 1)])
def test_selective_scan(kind, T, lens, D, N, G):
    import gated_delta_rule_scan_amd as gdn

    r = Rng(42)
    kw = _ssm_inputs(r, kind, (T,), D, N, G, True, True, True, True)
    s = r.t(len(lens), D, N)
    _compare(lambda out: gdn.selective_scan(**kw, state_in=s, seq_offsets=offsets(lens), out=out), kw["x"], slice(0, sum(lens)))


def _index(B, slots):
    """Slots of B rows, a third of them no slot; and the rows that have one."""
    torch = _torch()
    idx = np.arange(B, dtype=np.int32)
    idx[::3] = [(-1, slots, 2 ** 31 - 1, -2 ** 31)[i % 4] for i in range(len(idx[::3]))]
    used = torch.from_numpy(np.flatnonzero((idx >= 0) & (idx < slots))).cuda()
    return torch.from_numpy(idx).cuda(), used


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,D", [(1, 64), (7, 33), (40, 2048), (300, 1)])
def test_conv_step(kind, B, D):
    import gated_delta_rule_scan_amd as gdn

    r = Rng(43)
    x, w, pool = r.t(B, D, kind=kind), r.t(D, 4), r.t(B + 2, 3, D, kind=kind)
    index, used = _index(B, B + 2)

    def call(out):
        s = pool.clone()
        return gdn.causal_conv_step(x, w, None, s, state_index=index, out=out), s

    _compare(call, x, used)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,N,G", [(1, 64, 16, 1), (7, 33, 5, 3), (40, 2048, 16, 1), (9, 600, 256, 2), (100, 1, 1, 1)])
def test_selective_step(kind, B, D, N, G):
    import gated_delta_rule_scan_amd as gdn

    r = Rng(44)
    kw = _ssm_inputs(r, kind, (B,), D, N, G, True, True, True, True)
    pool = r.t(B + 2, D, N)
    index, used = _index(B, B + 2)

    def call(out):
        s = pool.clone()
        return gdn.selective_step(**kw, state=s, state_index=index, out=out), s

    _compare(call, kw["x"], used)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 12, 128, 128), (7, 3, 64, 128), (5, 4, 128, 64), (60, 16, 64, 64)])
@pytest.mark.parametrize("epilogue", [False, True])
def test_delta_step(kind, B, H, dk, dv, epilogue):
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(45)
    q, k, v = r.t(B, H, dk, kind=kind), r.t(B, H, dk, kind=kind), r.t(B, H, dv, kind=kind)
    la, beta = -r.t(B, H).abs(), torch.sigmoid(r.t(B, H))
    gate, nw = (r.t(B, H, dv, kind=kind), r.t(dv)) if epilogue else (None, None)
    pool = r.t(B + 2, H, dv, dk)
    index, used = _index(B, B + 2)

    def call(out):
        s = pool.clone()
        return gdn.delta_step(q, k, v, la, beta, s, index, gate=gate, norm_weight=nw, out=out), s

    _compare(call, v, used, dtype=torch.float32)


def test_traced_ops():
    """The torch.ops forms, which make their outputs."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    gdn.register_torch_ops()
    r = Rng(46)
    B, D, N, H, d, T = 6, 72, 16, 2, 64, 500
    index, used = _index(B, B)
    rest = torch.ones(B, dtype=torch.bool, device="cuda")
    rest[used] = False
    x, w = r.t(B, D, kind="bf16"), r.t(D, 4)
    _poison(x.shape, x.dtype)
    y = torch.ops.gdn.causal_conv_step(x, w, None, r.t(B, 3, D, kind="bf16"), "silu", index)
    assert (y[rest] == 0).all() and torch.isfinite(y).all()
    kw = _ssm_inputs(r, "bf16", (B,), D, N, 1, True, True, True, True)
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")
    state = r.t(B, D, N)
    _poison(x.shape, x.dtype)
    y = torch.ops.gdn.selective_step(*(kw[k] for k in names), True, state, index)
    assert (y[rest] == 0).all() and torch.isfinite(y).all()
    q, la, S = r.t(B, H, d), -r.t(B, H).abs(), r.t(B, H, d, d)
    _poison(q.shape, q.dtype)
    o = torch.ops.gdn.delta_step(q, q, q, la, torch.sigmoid(la), S, index, True, False, None, None, 1e-6)
    assert (o[rest] == 0).all() and torch.isfinite(o).all()
    off = offsets([100, 30])
    x = r.t(T, D, kind="bf16")
    _poison(x.shape, x.dtype)
    y, _ = torch.ops.gdn.causal_conv(x, w, None, None, "silu", off)
    assert (y[130:] == 0).all() and torch.isfinite(y).all()
    kw = _ssm_inputs(r, "bf16", (T,), D, N, 1, True, True, True, True)
    _poison(x.shape, x.dtype)
    y, _ = torch.ops.gdn.selective_scan(*(kw[k] for k in names), True, None, off)
    assert (y[130:] == 0).all() and torch.isfinite(y).all()


@pytest.mark.parametrize("name", ["conv", "scan", "conv step", "step", "delta step"])
def test_captured(name):
    """Captured and replayed with the slots and offsets changed in place: zeros follow the rows without a sequence."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    r = Rng(47)
    B, D, N, H, d, T = 6, 72, 16, 2, 64, 500
    kind = "bf16"
    index, off = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    x, w, px = r.t(B, D, kind=kind), r.t(D, 4), r.t(T, D, kind=kind)
    tok, prompt = (_ssm_inputs(r, kind, lead, D, N, 1, True, True, True, True) for lead in ((B,), (T,)))
    q, la, beta = r.t(B, H, d, kind=kind), -r.t(B, H).abs(), torch.sigmoid(r.t(B, H))
    cs, hs, S = r.t(B, 3, D, kind=kind), r.t(B, D, N), r.t(B, H, d, d)
    call = {"conv": lambda out: gdn.causal_conv(px, w, seq_offsets=off, out=out)[0],
            "scan": lambda out: gdn.selective_scan(**prompt, seq_offsets=off, out=out)[0],
            "conv step": lambda out: gdn.causal_conv_step(x, w, None, cs, state_index=index, out=out),
            "step": lambda out: gdn.selective_step(**tok, state=hs, state_index=index, out=out),
            "delta step": lambda out: gdn.delta_step(q, q, q, la, beta, S, index, out=out)}[name]
    start = [t.clone() for t in (cs, hs, S)]

    def reset():
        for t, s in zip((cs, hs, S), start):
            t.copy_(s)

    def choose(i):
        index.copy_(torch.tensor([[0, 1, 2, 3, 4, 5], [-1, 3, 6, 0, 1, -9], [5, -1, -1, -1, -1, 4]][i], dtype=torch.int32))
        off.copy_(torch.tensor([[0, 200, 500], [0, 0, 77], [0, 130, 131]][i], dtype=torch.int32))

    choose(0)
    call(None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = call(None)
    for i in (0, 1, 2, 1):
        choose(i)
        reset()
        want = call(torch.zeros_like(y))
        y.fill_(float("nan"))
        reset()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), f"choice {i}"
