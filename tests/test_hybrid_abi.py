"""The paged cache's, the attention step's and the seam's C ABI and binding on
the host (no kernel runs here): structure layouts, every argument check, the
launch-failure path of valid calls on a machine without a GPU, the oracle's
formats."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import gated_delta_rule_scan_amd as gdn
from test_layer_abi import HIP, INVALID, OK, ROOT, UNSUPPORTED, addr, no_gpu

STRUCTS = ("gdn_kv_problem_t", "gdn_attention_problem_t", "gdn_norm_problem_t")
ENUMS = ("GDN_KV_F32", "GDN_KV_BF16", "GDN_KV_MXFP8", "GDN_KV_MXFP4", "GDN_LAYER_OPT_ZERO_UNUSED")
ZERO = gdn.GDN_LAYER_OPT_ZERO_UNUSED


def test_struct_layouts_match_c(tmp_path):
    lines = []
    for s in STRUCTS:
        lines.append(f'printf("%zu\\n", sizeof({s}));')
        lines += [f'printf("%zu\\n", offsetof({s}, {f}));' for f, *_ in getattr(gdn, s)._fields_]
    lines += [f'printf("%d\\n", {e});' for e in ENUMS]
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gdn.h"\nint main(void) {' + "\n".join(lines) + "return 0; }")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", f"-I{os.path.join(ROOT, 'include')}", str(prog), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    want = []
    for s in STRUCTS:
        S = getattr(gdn, s)
        want += [ctypes.sizeof(S)] + [getattr(S, f).offset for f, *_ in S._fields_]
    assert got == want + [getattr(gdn, e) for e in ENUMS]


def _split(over, fields, args):
    a = dict(args)
    f = dict(fields)
    f.update({k: v for k, v in over.items() if k not in a})
    a.update({k: v for k, v in over.items() if k in a})
    return f, a


def kv(read=False, **over):
    f = dict(B=2, T=30, Hk=4, d=128, pages=100, page=16, table_width=5, dtype=1, format=1, page_table=addr(6), start=addr(7))
    for r in ("k", "v"):
        f[r + "_stride_b"], f[r + "_stride_t"], f[r + "_stride_h"] = 30 * 512, 512, 128
    f, a = _split(over, f, dict(k=addr(0), v=addr(1), k_cache=addr(2), v_cache=addr(3), k_scales=addr(4), v_scales=addr(5)))
    p = gdn.gdn_kv_problem_t(**f)
    if read:
        return gdn.gdn_kv_read(p, a["k_cache"], a["v_cache"], a["k_scales"], a["v_scales"], a["k"], a["v"])
    return gdn.gdn_kv_write(p, a["k"], a["v"], a["k_cache"], a["v_cache"], a["k_scales"], a["v_scales"])


def attention(**over):
    f = dict(B=2, Hq=8, Hk=4, d=128, pages=100, page=16, table_width=5, q_stride_b=1024, q_stride_h=128, out_stride_b=1024,
             out_stride_h=128, dtype=1, format=1, scale=0.1, page_table=addr(6), lengths=addr(7), workspace=addr(9),
             workspace_bytes=1 << 33)
    f, a = _split(over, f, dict(q=addr(0), k_cache=addr(2), v_cache=addr(3), k_scales=addr(4), v_scales=addr(5), out=addr(1),
                                lse=addr(8)))
    return gdn.gdn_attention_step(gdn.gdn_attention_problem_t(**f), a["q"], a["k_cache"], a["v_cache"], a["k_scales"],
                                  a["v_scales"], a["out"], a["lse"])


def norm_problem(**over):
    f = dict(B=2, T=30, D=64, gate_stride_b=64, dtype=1, residual_scale=1.0, eps=1e-6, gate=addr(10), post_weight=addr(11),
             weight=addr(12), workspace=addr(13), workspace_bytes=1 << 33)
    for r in ("x", "y", "h", "n", "dx", "dy"):
        f[r + "_stride_b"], f[r + "_stride_t"] = 30 * 64, 64
    f.update(over)
    return gdn.gdn_norm_problem_t(**f)


ROWS = dict(x=addr(0), y=addr(1), h=addr(2), n=addr(3))
GRADS = dict(dx=addr(4), dy=addr(5), dgate=addr(6), dpost_weight=addr(7), dweight=addr(8))


def norm(**over):
    a = {**ROWS, **{k: v for k, v in over.items() if k in ROWS}}
    p = norm_problem(**{k: v for k, v in over.items() if k not in ROWS})
    return gdn.gdn_norm_forward(p, a["x"], a["y"], a["h"], a["n"])


def norm_back(**over):
    names = {**ROWS, **GRADS}
    a = {**names, **{k: v for k, v in over.items() if k in names}}
    p = norm_problem(**{k: v for k, v in over.items() if k not in names})
    return gdn.gdn_norm_backward(p, a["x"], a["y"], a["h"], a["n"], a["dx"], a["dy"], a["dgate"], a["dpost_weight"], a["dweight"])


def test_null_problems_are_invalid():
    L = gdn.lib()
    x = addr(0)
    assert L.gdn_kv_write(None, x, x, x, x, x, x) == INVALID
    assert L.gdn_kv_read(None, x, x, x, x, x, x) == INVALID
    assert L.gdn_attention_step(None, x, x, x, x, x, x, x) == INVALID
    assert L.gdn_norm_forward(None, x, x, x, x) == INVALID
    assert L.gdn_norm_backward(None, x, x, x, x, x, x, x, x, x) == INVALID
    assert L.gdn_attention_workspace_bytes(None) == 0 and L.gdn_norm_workspace_bytes(None) == 0


CACHE_BAD = [  # sizes, pools and tables, of every call with a cache
    (dict(B=0), INVALID), (dict(B=1 << 31), INVALID), (dict(Hk=0), INVALID), (dict(d=0), INVALID), (dict(pages=0), INVALID),
    (dict(pages=1 << 31), INVALID), (dict(page=0), INVALID), (dict(table_width=0), INVALID), (dict(table_width=1 << 31), INVALID),
    (dict(format=-1), INVALID), (dict(format=4), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(dtype=0), UNSUPPORTED),
    (dict(format=0), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=512), UNSUPPORTED), (dict(page=8), UNSUPPORTED),
    (dict(page=2048), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(B=1 << 20, table_width=1 << 20), UNSUPPORTED),
    (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID), (dict(k_cache=addr(2) + 8), INVALID),
    (dict(v_cache=addr(3) + 4), INVALID), (dict(format=2, k_scales=None), INVALID), (dict(format=3, v_scales=None), INVALID),
    (dict(format=2, k_scales=addr(4) + 2), INVALID), (dict(format=2, v_scales=addr(5) + 1), INVALID),
    (dict(page_table=None), INVALID), (dict(page_table=addr(6) + 2), INVALID),
]


@pytest.mark.parametrize("over,status", CACHE_BAD)
def test_caches_that_are_refused(over, status):
    assert kv(**over) == status
    assert kv(read=True, **over) == status
    assert attention(**over) == status


KV_BAD = [
    (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=addr(0) + 1), INVALID),
    (dict(start=addr(7) + 2), INVALID), (dict(seq_offsets=addr(8) + 1), INVALID), (dict(k_stride_t=-1), INVALID),
    (dict(v_stride_h=-128), INVALID), (dict(v_stride_b=1 << 62), INVALID), (dict(options=1), INVALID), (dict(options=512), INVALID),
    (dict(B=1 << 12, T=1 << 20), UNSUPPORTED),
]


@pytest.mark.parametrize("over,status", KV_BAD)
def test_rows_of_a_cache_that_are_refused(over, status):
    assert kv(**over) == status
    assert kv(read=True, **over) == status


@pytest.mark.parametrize("over", [
    dict(k_cache=addr(0)), dict(v_cache=addr(1)), dict(v_cache=addr(2)), dict(v_cache=addr(2) + 99 * 16 * 512 * 2),
    dict(k_cache=addr(6)), dict(v_cache=addr(7)), dict(format=2, k_scales=addr(2)), dict(format=2, v_scales=addr(4)),
    dict(format=3, v_scales=addr(1)), dict(seq_offsets=addr(3)), dict(options=ZERO)])
def test_writes_that_overlap_are_refused(over):
    assert kv(**over) == INVALID


@pytest.mark.parametrize("over", [
    dict(k=addr(1)), dict(k=addr(2)), dict(v=addr(3) + 1000), dict(k=addr(6)), dict(v=addr(7)), dict(format=2, v=addr(4)),
    dict(k_stride_t=500), dict(v_stride_b=512), dict(k_stride_h=0), dict(seq_offsets=addr(0))])
def test_reads_that_overlap_are_refused(over):
    assert kv(read=True, **over) == INVALID


@no_gpu
@pytest.mark.parametrize("over", [dict(), dict(start=None), dict(format=2), dict(format=3), dict(dtype=0, format=0),
                                  dict(dtype=0, format=3), dict(seq_offsets=addr(8)), dict(page=1024), dict(d=64), dict(d=256, k_stride_h=256,
                                  v_stride_h=256, k_stride_t=1024, v_stride_t=1024, k_stride_b=1 << 20, v_stride_b=1 << 20),
                                  dict(k=addr(0) + 2), dict(v=addr(0) + 8 * 256, k_stride_t=1536, v_stride_t=1536,
                                                            k_stride_b=1536 * 30, v_stride_b=1536 * 30)])
def test_valid_rows_reach_the_launch(over):
    assert kv(**over) == HIP
    assert kv(read=True, **over) == HIP
    assert kv(read=True, options=ZERO, **over) == HIP


def test_no_rows_are_ok():
    assert kv(T=0, k=None, v=None) == OK and kv(read=True, T=0, k=None, v=None) == OK
    # rows of inputs may repeat (a row for every head, say)
    if not os.path.exists("/dev/kfd"):
        assert kv(k_stride_h=0, v_stride_t=0) == HIP


ATTENTION_BAD = [
    (dict(Hq=0), INVALID), (dict(Hq=6), INVALID), (dict(Hq=1 << 17, Hk=1), UNSUPPORTED), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(lengths=None), INVALID), (dict(q=addr(0) + 1), INVALID), (dict(out=addr(1) + 1), INVALID),
    (dict(lse=addr(8) + 2), INVALID), (dict(lengths=addr(7) + 1), INVALID), (dict(q_stride_b=-1), INVALID),
    (dict(out_stride_h=-1), INVALID), (dict(q_stride_h=1 << 41), INVALID), (dict(out_stride_h=64), INVALID),
    (dict(out_stride_b=0), INVALID), (dict(out=addr(0)), INVALID), (dict(out=addr(2)), INVALID), (dict(out=addr(3)), INVALID),
    (dict(out=addr(6)), INVALID), (dict(out=addr(7)), INVALID), (dict(lse=addr(1)), INVALID), (dict(lse=addr(0)), INVALID),
    (dict(lse=addr(3)), INVALID), (dict(format=2, out=addr(4)), INVALID), (dict(format=3, lse=addr(5)), INVALID),
    (dict(lse=addr(6)), INVALID),
]


@pytest.mark.parametrize("over,status", ATTENTION_BAD)
def test_attention_rejects(over, status):
    assert attention(**over) == status


@no_gpu
@pytest.mark.parametrize("over", [dict(), dict(lse=None), dict(format=2), dict(format=3), dict(dtype=0, format=0), dict(dtype=0, format=2),
                                  dict(Hq=128, Hk=1, q_stride_b=128 * 128, out_stride_b=128 * 128), dict(window=5, sinks=3), dict(q_stride_b=0, q_stride_h=0),
                                  dict(out=addr(0) + 2048, q_stride_b=2048, out_stride_b=2048), dict(page=1024, table_width=4096)])
def test_valid_attention_reaches_the_launch(over):
    assert attention(**over) == HIP


NORM_BAD = [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(D=0), INVALID), (dict(T=1 << 31), INVALID), (dict(D=16385, gate_stride_b=0), UNSUPPORTED),
    (dict(B=1 << 16, T=1 << 16), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(options=1), INVALID), (dict(options=ZERO | 2), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(residual_scale=float("inf")), INVALID), (dict(residual_scale=float("nan")), INVALID), (dict(gate_stride_b=63), INVALID),
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(n=None), INVALID), (dict(weight=None), INVALID),
    (dict(x=addr(0) + 1), INVALID), (dict(y=addr(1) + 1), INVALID), (dict(n=addr(3) + 1), INVALID), (dict(gate=addr(10) + 2), INVALID),
    (dict(post_weight=addr(11) + 1), INVALID), (dict(weight=addr(12) + 3), INVALID), (dict(seq_offsets=addr(14) + 2), INVALID),
    (dict(x_stride_t=-1), INVALID), (dict(y_stride_b=-5), INVALID), (dict(h_stride_t=1 << 41), INVALID),
]


@pytest.mark.parametrize("over,status", NORM_BAD)
def test_norm_rejects(over, status):
    assert norm(**over) == status
    assert norm_back(**over) == status


@pytest.mark.parametrize("over", [dict(h=None, n=None, weight=None), dict(h=addr(1)), dict(n=addr(0)), dict(n=addr(2)), dict(h=addr(10)),
                                  dict(n=addr(11)), dict(n=addr(12)), dict(h=addr(0) + 64), dict(h_stride_t=32), dict(n_stride_b=64),
                                  dict(h=addr(0), h_stride_t=65, h_stride_b=65 * 30), dict(seq_offsets=addr(2))])
def test_norm_forward_rejects(over):
    assert norm(**over) == INVALID


@pytest.mark.parametrize("over", [dict(dx=addr(0)), dict(dx=addr(3)), dict(dy=addr(2)), dict(dy=addr(4)), dict(dgate=addr(10)),
                                  dict(dgate=addr(8)), dict(dweight=addr(12)), dict(dpost_weight=addr(5)), dict(dweight=addr(8) + 2),
                                  dict(dx=addr(2), dx_stride_t=70), dict(dy_stride_t=8), dict(workspace=None), dict(workspace=addr(13) + 64),
                                  dict(workspace=addr(4)), dict(workspace=addr(2)), dict(workspace=addr(8)), dict(gate=None),
                                  dict(post_weight=None), dict(dx=addr(4) + 1), dict(dgate=addr(6) + 2),
                                  dict(y=None, gate=None, post_weight=None, dgate=None, dpost_weight=None)])
def test_norm_backward_rejects(over):
    assert norm_back(**over) == INVALID


def test_norm_workspace():
    size = lambda **k: gdn.gdn_norm_workspace_bytes(norm_problem(**k))
    assert size() > 0 and size(weight=None) == size(gate=None) == size() // 3 * 2
    assert size(gate=None, post_weight=None, weight=None) == 0 and size(D=20000) == 0 and size(eps=-1.0) == 0
    assert size(seq_offsets=addr(14)) > 0
    assert norm_back(workspace_bytes=size() - 1) == gdn.GDN_ERR_WORKSPACE_TOO_SMALL


@no_gpu
@pytest.mark.parametrize("over", [dict(), dict(gate=None, dgate=None), dict(post_weight=None, dpost_weight=None), dict(gate_stride_b=0),
                                  dict(y=None, gate=None, post_weight=None, dy=None, dgate=None, dpost_weight=None),
                                  dict(weight=None, n=None, dweight=None), dict(seq_offsets=addr(14)), dict(options=ZERO), dict(D=33, gate_stride_b=33),
                                  dict(dgate=None, dpost_weight=None, dweight=None, workspace=None), dict(dx=addr(2)),
                                  dict(dx=None, dy=None), dict(h=None), dict(D=16384, x_stride_t=16384, y_stride_t=16384, h_stride_t=16384,
                                  n_stride_t=16384, dx_stride_t=16384, dy_stride_t=16384, B=1, gate_stride_b=0)])
def test_valid_norms_reach_the_launch(over):
    assert norm_back(**over) == HIP
    if "dx" not in over:
        assert norm(**{k: v for k, v in over.items() if k not in GRADS}) == HIP


@no_gpu
def test_in_place_norms_reach_the_launch():
    assert norm(h=addr(0)) == HIP and norm(h=addr(0), x_stride_t=80, h_stride_t=80, x_stride_b=5000, h_stride_b=5000) == HIP


def test_no_rows_of_a_norm_are_ok():
    assert norm(T=0, x=None, y=None, h=None, n=None) == OK
    assert norm_back(T=0, dgate=None, dpost_weight=None, dweight=None) == OK


# ---- the binding ----

def test_binding_refuses():
    import torch

    z = torch.zeros
    q, pools, table, lens = z(2, 4, 64), (z(3, 2, 16, 64), z(3, 2, 16, 64)), z(2, 2, dtype=torch.int32), z(2, dtype=torch.int32)
    for call in (lambda: gdn.kv_write(q, q, pools, table), lambda: gdn.attention_step(q, pools, table, lens),
                 lambda: gdn.kv_read(pools, table, 3), lambda: gdn.residual_norm(q, q, weight=z(64)),
                 lambda: gdn.residual_norm_backward(q, q, q, q, weight=z(64))):
        with pytest.raises(ValueError):  # host tensors
            call()
    for call in (lambda: gdn.kv_write(q.half(), q.half(), pools, table), lambda: gdn.attention_step(q.double(), pools, table, lens),
                 lambda: gdn.kv_read(pools, table, 3, dtype=torch.float16), lambda: gdn.residual_norm(q.half(), q.half())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(TypeError):
        gdn.residual_norm([1.0])


def test_kv_cache():
    import torch

    c = gdn.kv_cache(5, 2, 16, 64, device="cpu")
    assert c.k.shape == c.v.shape == (5, 2, 16, 64) and c.k.dtype == torch.bfloat16 and c.k_scales is None
    assert gdn.kv_cache(1, 1, 1024, 256, "float32", device="cpu").v.dtype == torch.float32
    c = gdn.kv_cache(5, 2, 32, 128, "mxfp8", device="cpu")
    assert c.k.dtype == torch.float8_e4m3fn and c.k.shape[-1] == 128 and c.v_scales.shape == (5, 2, 32, 4)
    c = gdn.kv_cache(5, 2, 32, 128, "mxfp4", device="cpu")
    assert c.k.dtype == torch.uint8 and c.k.shape[-1] == 64 and c.k_scales.dtype == torch.uint8 and not c.k.any()
    for bad in (dict(format="int8"), dict(d=96), dict(page=24), dict(page=8), dict(page=2048)):
        with pytest.raises(ValueError):
            gdn.kv_cache(**{**dict(pages=1, heads=1, page=16, d=64, device="cpu"), **bad})


def test_custom_ops_trace_with_fake_tensors():
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode

    gdn.register_torch_ops()
    with FakeTensorMode():
        e = lambda *s, **k: torch.empty(s, device="cuda", **k)
        i = lambda *s: e(*s, dtype=torch.int32)
        k, pool = e(2, 30, 4, 64), e(9, 4, 16, 64)
        torch.ops.gdn.kv_write(k, k, pool, pool, None, None, i(2, 3), None, None)
        a, b = torch.ops.gdn.kv_read(pool, pool, None, None, i(2, 3), 7, None, None, torch.float32)
        assert a.shape == b.shape == (2, 7, 4, 64) and a.dtype == torch.float32
        codes, sc = e(9, 4, 16, 32, dtype=torch.uint8), e(9, 4, 16, 2, dtype=torch.uint8)
        a, b = torch.ops.gdn.kv_read(codes, codes, sc, sc, i(2, 3), 7, None, i(3), torch.bfloat16)
        assert a.shape == (7, 4, 64) and a.dtype == torch.bfloat16
        y, lse = torch.ops.gdn.attention_step(e(2, 8, 64), pool, pool, None, None, i(2, 3), i(2), None, 0, 0)
        assert y.shape == (2, 8, 64) and lse.shape == (2, 8) and lse.dtype == torch.float32
        x, w = e(2, 30, 64, dtype=torch.bfloat16), e(64)
        h, n = torch.ops.gdn.residual_norm(x, x, e(2, 64), None, w, 1.0, 1e-6, None)
        assert h.shape == n.shape == x.shape and n.dtype == torch.bfloat16
        g = torch.ops.gdn.residual_norm_backward(x, x, x, x, e(2, 64), None, w, 1.0, 1e-6, None)
        assert [t.shape for t in g] == [x.shape, x.shape, (2, 64), (0,), (64,)] and g[2].dtype == torch.float32


# ---- the oracle's formats ----

def test_oracle_formats():
    import hybrid_oracle as oracle

    assert oracle.E4M3[-1] == 448 and oracle.E4M3[1] == 2.0 ** -9 and (np.diff(oracle.E4M3) > 0).all()
    x = np.zeros((1, 64))
    x[0, 0], x[0, 1], x[0, 2], x[0, 32] = 448, 18.5, 17.0, 449  # 18.5 lies nearer 18; 17 half-way: to 16 (even)
    c, s = oracle.encode(x, "mxfp8")
    assert list(s[0]) == [127, 128]
    v = oracle.decode(c, s, "mxfp8")
    assert list(v[0, :3]) == [448, 18, 16] and v[0, 32] == 448
    x = np.zeros((1, 32))
    x[0, :6] = [6, 2.5, -3.5, 5, 0.25, 0.75]
    c, s = oracle.encode(x, "mxfp4")
    assert s[0, 0] == 127 and list(oracle.decode(c, s, "mxfp4")[0, :6]) == [6, 2, -4, 4, 0, 1]
    assert oracle.encode(x * 0, "mxfp4")[1][0, 0] == 17 and oracle.encode(x + np.inf, "mxfp8")[1][0, 0] == 255


def test_oracle_gradients_against_differences():
    import hybrid_oracle as oracle

    g = np.random.default_rng(3)
    R, D = 5, 7
    x, y, gate, post, w, dh, dn = (g.standard_normal(s) for s in ((R, D), (R, D), (R, D), (D,), (D,), (R, D), (R, D)))
    got = oracle.seam_backward(dh, dn, x, y, gate, post, w, 0.7, 1e-3, [(i, i + 1) for i in range(R)])

    def loss(x, y, gate, post, w):
        (h, _), (n, _) = oracle.seam(x, y, gate, post, w, 0.7, 1e-3)
        return (h * dh).sum() + (n * dn).sum()

    args = [x, y, gate, post, w]
    for i, name in enumerate(("dx", "dy", "dgate", "dpost", "dweight")):
        r = g.standard_normal(args[i].shape)
        at = lambda s: loss(*(a + s * r if j == i else a for j, a in enumerate(args)))
        slope = (8 * (at(1e-3) - at(-1e-3)) - (at(2e-3) - at(-2e-3))) / 12e-3
        assert abs(slope - (got[name][0] * r).sum()) < 1e-7
