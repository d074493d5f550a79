"""The layer operators' C ABI and binding on the host (no kernel runs here):
structure layouts, every argument check, and the launch-failure path of valid
calls on a machine without a GPU."""
import ctypes
import os
import subprocess

import pytest

import gated_delta_rule_scan_amd as gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = ("gdn_conv_problem_t", "gdn_ssm_problem_t", "gdn_rotary_problem_t", "gdn_step_problem_t")
OK, INVALID, UNSUPPORTED, HIP = gdn.GDN_OK, gdn.GDN_ERR_INVALID_ARGUMENT, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_HIP
no_gpu = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU is present: the launch would succeed")


def test_struct_layouts_match_c(tmp_path):
    lines = []
    for s in STRUCTS:
        lines.append(f'printf("%zu\\n", sizeof({s}));')
        lines += [f'printf("%zu\\n", offsetof({s}, {f}));' for f, *_ in getattr(gdn, s)._fields_]
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gdn.h"\nint main(void) {' + "\n".join(lines)
                    + 'printf("%d %d %d %d %d\\n", GDN_ACT_NONE, GDN_ACT_SILU, GDN_SSM_OPT_SOFTPLUS, '
                      'GDN_ROTARY_OPT_INTERLEAVED, GDN_ROTARY_OPT_INVERSE); return 0; }')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", f"-I{os.path.join(ROOT, 'include')}", str(prog), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    want = []
    for s in STRUCTS:
        S = getattr(gdn, s)
        want += [ctypes.sizeof(S)] + [getattr(S, f).offset for f, *_ in S._fields_]
    want += [gdn.GDN_ACT_NONE, gdn.GDN_ACT_SILU, gdn.GDN_SSM_OPT_SOFTPLUS, gdn.GDN_ROTARY_OPT_INTERLEAVED,
             gdn.GDN_ROTARY_OPT_INVERSE]
    assert got == want


# Fake, well-aligned device addresses: validation never dereferences them.
BASE, GAP = 1 << 40, 1 << 34


def addr(i):
    return BASE + i * GAP


def conv(step=False, **over):
    f = dict(B=2, T=300, D=64, x_stride_b=300 * 64, x_stride_t=64, out_stride_b=300 * 64, out_stride_t=64, slots=2,
             dtype=gdn.GDN_DTYPE_BF16, width=4, activation=1)
    if step:
        f.update(x_stride_b=64, out_stride_b=64)
    a = dict(x=addr(0), weight=addr(1), bias=addr(2), state_in=addr(3), state_out=addr(4), out=addr(5))
    f.update({k: v for k, v in over.items() if k not in a})
    a.update({k: v for k, v in over.items() if k in a})
    p = gdn.gdn_conv_problem_t(**f)
    if step:
        return gdn.gdn_conv_step(p, a["x"], a["weight"], a["bias"], a["state_out"], a["out"])
    return gdn.gdn_conv_forward(p, a["x"], a["weight"], a["bias"], a["state_in"], a["state_out"], a["out"])


def ssm(step=False, **over):
    f = dict(B=2, T=300, D=64, N=16, G=2, slots=2, dtype=gdn.GDN_DTYPE_BF16, options=1, z=addr(6), dt_bias=addr(7),
             skip=addr(8), workspace=addr(12), workspace_bytes=1 << 30)
    for r in ("x", "dt", "z", "out"):
        f[r + "_stride_b"], f[r + "_stride_t"] = (64, 0) if step else (300 * 64, 64)
    for r in ("b", "c"):
        f[r + "_stride_b"], f[r + "_stride_t"] = (32, 0) if step else (300 * 32, 32)
    a = dict(x=addr(0), dt=addr(1), A=addr(2), Bm=addr(3), Cm=addr(4), state_in=addr(9), state_out=addr(10), out=addr(5))
    f.update({k: v for k, v in over.items() if k not in a})
    a.update({k: v for k, v in over.items() if k in a})
    p = gdn.gdn_ssm_problem_t(**f)
    if step:
        return gdn.gdn_ssm_step(p, a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["state_out"], a["out"])
    return gdn.gdn_ssm_forward(p, a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["state_in"], a["state_out"], a["out"])


def rotary(**over):
    f = dict(B=2, T=30, Hq=4, Hk=2, d=128, rot=64, q_stride_b=30 * 1024, q_stride_t=1024, q_stride_h=128,
             k_stride_b=30 * 1024, k_stride_t=1024, k_stride_h=128, q_out_stride_b=30 * 512, q_out_stride_t=512,
             q_out_stride_h=128, k_out_stride_b=30 * 256, k_out_stride_t=256, k_out_stride_h=128,
             dtype=gdn.GDN_DTYPE_BF16, position_bits=64, axes=1, scale=1.0)
    # q and k beside each other in one projection's rows
    a = dict(q=addr(0), k=addr(0) + 512 * 2, inv_freq=addr(1), positions=addr(2), q_out=addr(3), k_out=addr(4))
    f.update({k: v for k, v in over.items() if k not in a})
    a.update({k: v for k, v in over.items() if k in a})
    if "section" in f:
        f["section"] = (ctypes.c_int32 * 4)(*f["section"])
    return gdn.gdn_rotary(gdn.gdn_rotary_problem_t(**f), a["q"], a["k"], a["inv_freq"], a["positions"], a["q_out"],
                          a["k_out"])


def step(**over):
    f = dict(B=2, H=3, dk=128, dv=64, slots=2, dtype=gdn.GDN_DTYPE_BF16)
    a = dict(q=addr(0), k=addr(1), v=addr(2), log_alpha=addr(3), beta=addr(4), state=addr(5), out=addr(6))
    f.update({k: v for k, v in over.items() if k not in a})
    a.update({k: v for k, v in over.items() if k in a})
    return gdn.gdn_step(gdn.gdn_step_problem_t(**f), a["q"], a["k"], a["v"], a["log_alpha"], a["beta"], a["state"],
                        a["out"])


def test_null_problems_are_invalid():
    L = gdn.lib()
    x = addr(0)
    assert L.gdn_conv_forward(None, x, x, x, x, x, x) == INVALID
    assert L.gdn_conv_step(None, x, x, x, x, x) == INVALID
    assert L.gdn_ssm_forward(None, x, x, x, x, x, x, x, x) == INVALID
    assert L.gdn_ssm_step(None, x, x, x, x, x, x, x) == INVALID
    assert L.gdn_rotary(None, x, x, x, x, x, x) == INVALID
    assert L.gdn_step(None, x, x, x, x, x, x, x) == INVALID


CONV_BAD = [
    (dict(B=0), INVALID), (dict(D=0), INVALID), (dict(T=-1), INVALID), (dict(B=1 << 31), INVALID),
    (dict(T=1 << 31), INVALID), (dict(activation=2), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(width=1), UNSUPPORTED),
    (dict(width=5), UNSUPPORTED), (dict(x_stride_t=-64), INVALID), (dict(out_stride_b=-1), INVALID),
    (dict(x_stride_b=1 << 62), INVALID), (dict(slots=3), INVALID), (dict(slots=0, state_index=addr(8)), INVALID),
    (dict(state_index=addr(8) + 2), INVALID), (dict(seq_offsets=addr(8) + 1, slots=2), INVALID),
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(out=None), INVALID), (dict(x=addr(0) + 1), INVALID),
    (dict(weight=addr(1) + 2), INVALID), (dict(bias=addr(2) + 1), INVALID), (dict(state_in=addr(3) + 1), INVALID),
    (dict(out=addr(0)), INVALID),                       # over the input
    (dict(out=addr(0) + 300 * 64 * 2), INVALID),        # over its second sequence
    (dict(out_stride_t=63), INVALID), (dict(out_stride_b=64), INVALID), (dict(out_stride_t=0), INVALID),  # rows that meet
    (dict(state_out=addr(0)), INVALID), (dict(state_out=addr(5)), INVALID), (dict(state_in=addr(5)), INVALID),
    (dict(state_out=addr(3) + 64), INVALID),            # half over the initial state
    (dict(state_out=addr(1)), INVALID), (dict(out=addr(1)), INVALID), (dict(out=addr(2)), INVALID),
]


@pytest.mark.parametrize("over,status", CONV_BAD)
def test_conv_rejects(over, status):
    assert conv(**over) == status
    if not any(k in over for k in ("T", "x_stride_t", "out_stride_t", "seq_offsets", "state_in", "out_stride_b", "x_stride_b")) \
            and over not in (dict(out=addr(0) + 300 * 64 * 2), dict(state_out=addr(3) + 64)):
        assert conv(step=True, **over) == status


def test_conv_step_needs_a_state():
    assert conv(step=True, state_out=None) == INVALID


def test_nothing_to_do_is_ok():
    assert conv(T=0, x=None, out=None, state_out=None) == OK
    assert ssm(T=0, x=None, dt=None, Bm=None, Cm=None, out=None, state_out=None) == OK
    assert rotary(T=0) == OK


@no_gpu
@pytest.mark.parametrize("over", [dict(), dict(state_out=addr(3)), dict(state_in=None), dict(state_in=None, state_out=None),
                                  dict(bias=None), dict(seq_offsets=addr(8)), dict(state_index=addr(8), slots=99),
                                  dict(x=addr(0) + 2, dtype=gdn.GDN_DTYPE_BF16),      # unaligned rows
                                  dict(x_stride_b=0), dict(T=0),
                                  # beside the input in one buffer of rows twice as wide
                                  dict(x_stride_t=128, x_stride_b=300 * 128, out_stride_t=128, out_stride_b=300 * 128,
                                       out=addr(0) + 128)])
def test_conv_valid_calls_reach_the_launch(over):
    assert conv(**over) == HIP


SSM_BAD = [
    (dict(B=0), INVALID), (dict(D=0), INVALID), (dict(N=0), INVALID), (dict(G=0), INVALID), (dict(G=3), INVALID),
    (dict(G=128, D=64), INVALID), (dict(N=257), UNSUPPORTED), (dict(dtype=5), UNSUPPORTED), (dict(options=2), INVALID),
    (dict(A=None), INVALID), (dict(x=None), INVALID), (dict(dt=None), INVALID), (dict(Bm=None), INVALID),
    (dict(Cm=None), INVALID), (dict(out=None), INVALID), (dict(slots=1), INVALID), (dict(z=addr(6) + 1), INVALID),
    (dict(dt_bias=addr(7) + 2), INVALID), (dict(skip=addr(8) + 3), INVALID), (dict(A=addr(2) + 1), INVALID),
    (dict(out=addr(0)), INVALID), (dict(out=addr(1)), INVALID), (dict(out=addr(3)), INVALID), (dict(out=addr(6)), INVALID),
    (dict(out=addr(2)), INVALID), (dict(out=addr(7)), INVALID), (dict(out=addr(10)), INVALID),
    (dict(state_out=addr(0)), INVALID), (dict(state_out=addr(2)), INVALID), (dict(state_out=addr(4)), INVALID),
    (dict(state_out=addr(10) + 2), INVALID), (dict(b_stride_b=-1), INVALID), (dict(c_stride_b=1 << 41), INVALID),
]


@pytest.mark.parametrize("over,status", SSM_BAD)
def test_ssm_rejects(over, status):
    assert ssm(**over) == status
    assert ssm(step=True, **over) == status


@pytest.mark.parametrize("over", [dict(T=-1), dict(T=1 << 31), dict(x_stride_t=-1), dict(state_in=addr(10) + 128),
                                  dict(state_in=addr(5)), dict(out_stride_t=32), dict(seq_offsets=addr(11) + 2), dict(workspace=None),
                                  dict(workspace=addr(12) + 128), dict(workspace=addr(0)), dict(workspace=addr(5)),
                                  dict(workspace=addr(9)), dict(workspace=addr(10)), dict(workspace=addr(2))])
def test_ssm_forward_rejects(over):
    assert ssm(**over) == INVALID


@pytest.mark.parametrize("name", ["x", "dt", "z", "b", "c", "out"])
def test_ssm_token_strides_are_bounded(name):
    assert ssm(T=300, **{name + "_stride_t": 1 << 26, name + "_stride_b": 1 << 36}) == UNSUPPORTED


def test_ssm_workspace():
    def size(packed=False, **k):
        p = gdn.gdn_ssm_problem_t(**dict(dict(B=1, T=4096, D=2048, N=16, G=1, dtype=1), **k))
        p.seq_offsets = addr(0) if packed else None
        return gdn.gdn_ssm_workspace_bytes(p)

    small = size()
    assert 0 < small and size(T=8192) >= small and size(packed=True) > 0
    assert size(T=0) == 0 and size(T=1) == 0 and size(T=36) == 0       # few tokens
    assert size(B=64) == 0                                             # enough sequences
    assert size(N=257) == 0 and size(dtype=7) == 0 and size(G=3) == 0  # unsupported, invalid
    assert ssm(workspace_bytes=4096) == gdn.GDN_ERR_WORKSPACE_TOO_SMALL


@no_gpu
@pytest.mark.parametrize("over", [dict(), dict(state_out=addr(9)), dict(state_in=None, state_out=None, slots=0),
                                  dict(z=None, dt_bias=None, skip=None), dict(seq_offsets=addr(11)),
                                  dict(state_index=addr(11), slots=7), dict(T=0), dict(N=256, b_stride_t=512, c_stride_t=512)])
def test_ssm_valid_calls_reach_the_launch(over):
    assert ssm(**over) == HIP
    if "state_out" not in over and "seq_offsets" not in over:
        assert ssm(step=True, **over) == HIP


ROTARY_BAD = [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hk=-1), INVALID), (dict(rot=0), INVALID),
    (dict(rot=63), INVALID), (dict(rot=130), INVALID), (dict(d=258), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(options=4), INVALID), (dict(position_bits=16), INVALID), (dict(axes=0), INVALID), (dict(axes=5), INVALID),
    (dict(axes=2, section=(16, 15, 0, 0)), INVALID), (dict(axes=2, section=(40, -8, 0, 0)), INVALID),
    (dict(axes=2, section=(16, 16, 0, 0), position_bits=0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(position0=1 << 60), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(q_out=None), INVALID), (dict(inv_freq=None), INVALID), (dict(positions=None), INVALID),
    (dict(inv_freq=addr(1) + 4), INVALID), (dict(positions=addr(2) + 4), INVALID), (dict(q=addr(0) + 1), INVALID),
    (dict(q_stride_t=-1), INVALID), (dict(q_out_stride_h=64), INVALID), (dict(q_out_stride_t=0), INVALID),
    (dict(q_out=addr(4)), INVALID), (dict(q_out=addr(0)), INVALID),          # the input, with other strides
    (dict(q_out=addr(1)), INVALID), (dict(k_out=addr(2)), INVALID), (dict(k_out=addr(0)), INVALID),
    (dict(B=1 << 20, T=1 << 20), UNSUPPORTED),
]


@pytest.mark.parametrize("over,status", ROTARY_BAD)
def test_rotary_rejects(over, status):
    assert rotary(**over) == status


FUSED = dict(q_out=addr(0), q_out_stride_b=30 * 1024, q_out_stride_t=1024, k_out=addr(0) + 1024, k_out_stride_b=30 * 1024,
             k_out_stride_t=1024)


@no_gpu
@pytest.mark.parametrize("over", [dict(), FUSED, dict(Hk=0, k=None, k_out=None), dict(Hq=2, **FUSED),
                                  dict(axes=3, section=(12, 10, 10, 0)), dict(position_bits=0, positions=None),
                                  dict(position_bits=32, positions=addr(2) + 4), dict(rot=20), dict(options=3)])
def test_rotary_valid_calls_reach_the_launch(over):
    assert rotary(**over) == HIP


STEP_BAD = [
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(dk=0), INVALID), (dict(dk=96), UNSUPPORTED),
    (dict(dv=32), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(options=1), INVALID), (dict(options=8), INVALID),
    (dict(slots=3), INVALID), (dict(slots=0, state_index=addr(9)), INVALID), (dict(B=1 << 20, H=1 << 20, slots=1 << 20), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(state=None), INVALID), (dict(out=None), INVALID), (dict(q=addr(0) + 8), INVALID),
    (dict(state=addr(5) + 4), INVALID), (dict(beta=addr(4) + 2), INVALID), (dict(gate=addr(7)), INVALID),
    (dict(gate=addr(7), norm_weight=addr(8), norm_eps=-1.0), INVALID), (dict(out=addr(0)), INVALID),
    (dict(out=addr(5)), INVALID), (dict(state=addr(1)), INVALID), (dict(gate=addr(6), norm_weight=addr(8)), INVALID),
    (dict(gate=addr(7), norm_weight=addr(5)), INVALID), (dict(state_index=addr(5)), INVALID),
]


@pytest.mark.parametrize("over,status", STEP_BAD)
def test_step_rejects(over, status):
    assert step(**over) == status


@no_gpu
@pytest.mark.parametrize("over", [dict(), dict(options=2 | 4), dict(gate=addr(7), norm_weight=addr(8), norm_eps=1e-6),
                                  dict(state_index=addr(9), slots=50)])
def test_step_valid_calls_reach_the_launch(over):
    assert step(**over) == HIP


# ---- the binding ----

def test_binding_rejects_host_tensors_and_types():
    import torch

    x, w = torch.zeros(2, 3, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError):
        gdn.causal_conv(x, w)
    with pytest.raises(TypeError):
        gdn.causal_conv(x.half(), w)
    with pytest.raises(TypeError):
        gdn.rotary(x.double()[None], None, torch.zeros(2, dtype=torch.float64))
    with pytest.raises(AttributeError):
        gdn.no_such_operator


def test_rotary_frequencies():
    import math

    import torch

    f, s = gdn.rotary_frequencies(8, base=100.0)
    assert f.dtype == torch.float64 and s == 1.0
    assert torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 100 ** -0.5, 100 ** -0.75], dtype=torch.float64), rtol=1e-15)
    assert torch.equal(gdn.rotary_frequencies(8, 100.0, "linear", 4.0)[0], f / 4)
    g, s = gdn.rotary_frequencies(8, 100.0, "base", 4.0)
    assert g[0] == 1.0 and math.isclose(float(g[-1]), float(f[-1]) / 4, rel_tol=1e-12) and s == 1.0
    g, s = gdn.rotary_frequencies(64, 10000.0, "parts", 8.0, original=4096, slow=1.0, fast=32.0)
    h = gdn.rotary_frequencies(64)[0]
    turns = 4096 * h / (2 * math.pi)
    assert torch.equal(g[turns >= 32], h[turns >= 32]) and torch.allclose(g[turns <= 1], h[turns <= 1] / 8, rtol=1e-15)
    between = (turns > 1) & (turns < 32)
    assert between.any() and ((g < h) & (g > h / 8))[between].all() and s == 0.1 * math.log(8.0) + 1.0
    assert torch.equal(gdn.rotary_frequencies(8, 100.0, "pairs", factors=[1, 2, 3, 4])[0], f / torch.tensor([1.0, 2, 3, 4]))
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, scaling="x"), dict(rot=8, factor=0.5), dict(rot=2, scaling="base"),
                dict(rot=8, scaling="pairs"), dict(rot=8, scaling="pairs", factors=[1.0]),
                dict(rot=8, scaling="parts", slow=3.0, fast=3.0)):
        with pytest.raises(ValueError):
            gdn.rotary_frequencies(**bad)


def test_custom_ops_trace_with_fake_tensors():
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode

    gdn.register_torch_ops()
    with FakeTensorMode():
        e = lambda *s, **k: torch.empty(s, device="cuda", **k)
        x = e(2, 30, 64, dtype=torch.bfloat16)
        y, s = torch.ops.gdn.causal_conv(x, e(64, 4), None, None, "silu", None)
        assert y.shape == x.shape and s.shape == (2, 3, 64) and s.dtype == torch.bfloat16
        off = e(6, dtype=torch.int32)
        y, s = torch.ops.gdn.causal_conv(x[0], e(64, 3), None, None, "none", off)
        assert y.shape == (30, 64) and s.shape == (5, 2, 64)
        B = e(2, 30, 1, 16, dtype=torch.bfloat16)
        y, h = torch.ops.gdn.selective_scan(x, x, e(64, 16), B, B, None, None, None, True, None, None)
        assert y.dtype == torch.bfloat16 and h.shape == (2, 64, 16) and h.dtype == torch.float32
        t = e(2, 64, dtype=torch.bfloat16)
        assert torch.ops.gdn.causal_conv_step(t, e(64, 4), None, e(2, 3, 64, dtype=torch.bfloat16), "silu", None).shape == (2, 64)
        Bt = e(2, 16, dtype=torch.bfloat16)
        assert torch.ops.gdn.selective_step(t, t, e(64, 16), Bt, Bt, None, None, None, True, e(2, 64, 16), None).shape == (2, 64)
        q = e(2, 30, 4, 64)
        a, b = torch.ops.gdn.rotary(q, q[:, :, :1], e(16, dtype=torch.float64), None, False, None, 1.0, False, 0)
        assert a.shape == q.shape and b.shape == (2, 30, 1, 64)
        o = torch.ops.gdn.delta_step(q[:, 0], q[:, 0], q[:, 0], e(2, 4), e(2, 4), e(2, 4, 64, 64), None, True, False, None,
                                     None, 1e-6)
        assert o.shape == (2, 4, 64) and o.dtype == torch.float32
