"""The largest batches of the cache, its attention and the seam on the GPU: more workgroups than one launch takes,
against the same rows in calls that need fewer; more sequences than are cut; workspaces of exactly the size that a call
asks for; lengths beyond a table whose pages are all there."""
import pytest

from layer_oracle import U
from test_gpu_hybrid import SeamCase, _attention_case, _check_attention, _expect, i32
from test_gpu_layer import _torch
from test_gpu_layer_together import G, _guarded

pytestmark = pytest.mark.gpu

MOST = ((1 << 32) - 1) // 256  # workgroups of 256 threads of one launch


def randn(seed, *shape):
    torch = _torch()
    return torch.randn(shape, dtype=torch.bfloat16, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))


def test_residual_norm_backward_of_more_gates_than_a_launch_takes():
    """65536 gates and a weight of 4096 channels: 8388736 workgroups of 512 threads in the sums' kernel."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    B, D = 65536, 4096
    x, y, dh, dn = (randn(s, B, D) for s in range(4))
    gate = torch.randn((B, D), device="cuda", generator=torch.Generator("cuda").manual_seed(9))
    weight = torch.linspace(0.5, 1.5, D, device="cuda")
    _, nn = gdn.residual_norm(x, y, gate=gate, weight=weight)
    mag = torch.zeros(D, dtype=torch.float64, device="cuda")
    for i in range(0, B, 8192):
        mag += (dn[i: i + 8192].double() * nn[i: i + 8192].double() / weight).abs().sum(0)
    halves = [gdn.residual_norm_backward(dh[i], dn[i], x[i], y[i], gate=gate[i], weight=weight)
              for i in (slice(0, B // 2), slice(B // 2, B))]
    got = gdn.residual_norm_backward(dh, dn, x, y, gate=gate, weight=weight, dx=dh)
    assert got[0].data_ptr() == dh.data_ptr() and got[3] is None
    for g, *h in zip(got[:3], *[p[:3] for p in halves]):
        assert torch.equal(g, torch.cat(h))
    # sums of 65536 products, in two orders: as many roundings in each at most, of no more than the sum of magnitudes
    # (1.01: that sum is taken from a rounded n)
    off = (got[4].double() - halves[0][4].double() - halves[1][4].double()).abs()
    assert (off <= 2 * (B + 64) * U * 1.01 * mag).all()


def test_rows_of_more_sequences_than_a_launch_takes():
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    B, D = MOST + 3, 8
    x, y, dn = (randn(s, B, D) for s in range(3))
    w = torch.linspace(0.5, 1.5, D, device="cuda")
    h, nn = gdn.residual_norm(x, y, weight=w)
    h1, n1 = gdn.residual_norm(x[None], y[None], weight=w)  # one sequence: its workgroups take many rows
    assert torch.equal(h, h1[0]) and torch.equal(nn, n1[0])
    got = gdn.residual_norm_backward(None, dn, x, y, weight=w)
    want = gdn.residual_norm_backward(None, dn[None], x[None], y[None], weight=w)
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[1][0])


def test_cache_rows_of_more_sequences_than_a_launch_takes():
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    B, page, d = MOST + 7, 16, 64
    k, v = randn(1, B, 1, d), randn(2, B, 1, d)
    at = torch.arange(B, dtype=torch.int32, device="cuda")
    table, start = (at // page)[:, None].contiguous(), at % page
    cache = gdn.kv_cache(-(-B // page), 1, page, d)
    gdn.kv_write(k, v, cache, table, start)
    assert torch.equal(cache.k.view(-1, 1, d)[:B], k) and torch.equal(cache.v.view(-1, 1, d)[:B], v)
    assert not cache.k.view(-1, d)[B:].any()
    back = gdn.kv_read(cache, table, 1, start)
    assert torch.equal(back[0][:, 0], k) and torch.equal(back[1][:, 0], v)


def test_attention_of_more_heads_than_a_launch_takes():
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    H, d, page = 128, 64, 16
    B = MOST // H + 30
    q = randn(1, B, H, d)
    cache = gdn.KVCache(randn(2, 5, H, page, d), randn(3, 5, H, page, d))
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None] % 5
    lens = torch.arange(B, dtype=torch.int32, device="cuda") % 17
    lse = torch.empty((B, H), device="cuda")
    y = gdn.attention_step(q, cache, table.contiguous(), lens, lse=lse)
    for i in (slice(0, B // 2), slice(B // 2, B)):
        part = torch.empty_like(lse[i])
        assert torch.equal(y[i], gdn.attention_step(q[i], cache, table[i].contiguous(), lens[i], lse=part))
        assert torch.equal(lse[i], part)


@pytest.mark.parametrize("kind,form", [("bf16", "bf16"), ("f32", "mxfp8")])
def test_attention_of_as_many_sequences_as_are_cut(kind, form):
    """1000 in a wide table: lengths in sixteen rounds of 64, long sequences in the first, a middle and the last."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    lens = [3, 40, 0, 17] * 250
    lens[5], lens[500], lens[999] = 3100, 2000, 5000
    q, cache, table, kv, vv = _attention_case(kind, form, lens, 4, 2, 64, 64, 0, 0, 32, width=100)
    lse = torch.empty((len(lens), 4), device="cuda")
    y = gdn.attention_step(q, cache, i32(table), i32(lens), lse=lse)
    _check_attention(y, lse, _expect(q, table, lens, kv, vv, 0.125, 0, 0, kind), kind)


@pytest.mark.parametrize("kind,form", [("bf16", "bf16"), ("f32", "mxfp8")])
def test_attention_of_a_thousand_sequences_in_a_wide_table(kind, form):
    """Not cut, short ones and one long one."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    lens = [3, 40, 0, 17] * 256 + [4100, 700]
    q, cache, table, kv, vv = _attention_case(kind, form, lens, 4, 2, 64, 64, 0, 0, 31, width=100)
    lse = torch.empty((len(lens), 4), device="cuda")
    y = gdn.attention_step(q, cache, i32(table), i32(lens), lse=lse)
    _check_attention(y, lse, _expect(q, table, lens, kv, vv, 0.125, 0, 0, kind), kind)


def _workspace(size):
    """(exactly that many bytes that hold NaN, the buffer with their guard zones)."""
    torch = _torch()
    ws, whole = _guarded(torch.full((size,), 255, dtype=torch.uint8, device="cuda"))
    assert ws.data_ptr() % 256 == 0
    return ws, whole


WORKSPACES = [
    # kind, form, lens, Hq, Hk, d, page, window, sinks, width
    ("bf16", "bf16", [1000], 12, 12, 128, 64, 0, 0, None),
    ("f32", "f32", [700, 0, 3000], 6, 2, 64, 16, 0, 0, None),
    ("bf16", "mxfp8", [5000, 1, 33, 600], 40, 1, 128, 64, 0, 0, 100),
    ("f32", "mxfp4", [2000, 40], 8, 2, 256, 16, 0, 0, 200),
    ("bf16", "bf16", [3000, 2500, 10], 34, 2, 256, 32, 900, 70, None),
    ("f32", "f32", [9000], 4, 4, 64, 32, 2500, 0, 400),
    ("bf16", "mxfp4", [600] * 70, 4, 2, 64, 64, 0, 0, 40),
]


@pytest.mark.parametrize("kind,form,lens,Hq,Hk,d,page,window,sinks,width", WORKSPACES)
def test_attention_keeps_to_its_workspace(kind, form, lens, Hq, Hk, d, page, window, sinks, width):
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    q, cache, table, kv, vv = _attention_case(kind, form, lens, Hq, Hk, d, page, window, sinks, len(lens) + d, width)
    forms = {"f32": 0, "bf16": 1, "mxfp8": 2, "mxfp4": 3}
    size = gdn.gdn_attention_workspace_bytes(gdn.gdn_attention_problem_t(
        B=len(lens), Hq=Hq, Hk=Hk, d=d, pages=len(kv), page=page, table_width=table.shape[1], window=window, sinks=sinks,
        dtype=forms[kind], format=forms[form]))
    assert size > 0
    ws, whole = _workspace(size)
    lse = torch.empty((len(lens), Hq), device="cuda")
    for _ in range(2):  # (the second call finds the first one's remains)
        y = gdn.attention_step(q, cache, i32(table), i32(lens), window=window, sinks=sinks, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        assert (whole[:G] == 0x5A).all() and (whole[-G:] == 0x5A).all()
        _check_attention(y, lse, _expect(q, table, lens, kv, vv, d ** -0.5, window, sinks, kind), kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("lens,D", [((2, 300), 136), ((5000,), 64), ([700, 0, 130], 1001), ([1] * 300, 250), ((1, 2000), 4003), ((3, 5), 16384)])
@pytest.mark.parametrize("gate,post,weight", [("sequence", True, True), ("channel", False, True), (None, True, False)])
def test_residual_norm_backward_keeps_to_its_workspace(kind, lens, D, gate, post, weight):
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    c = SeamCase(kind, lens, D, True, gate, post, weight, 1.0, "plain")
    packed = isinstance(lens, list)
    p = gdn.gdn_norm_problem_t(B=len(c.each), T=c.x.shape[0] if packed else lens[1] if len(lens) == 2 else 1, D=D,
                               gate_stride_b=D if gate == "sequence" else 0, dtype=int(kind == "bf16"), residual_scale=1.0, eps=1e-6)
    p.gate, p.post_weight, p.weight, p.seq_offsets = (1 << 20 if t is not None else None for t in (c.gate, c.post, c.weight, c.off))
    size = gdn.gdn_norm_workspace_bytes(p)
    assert size > 0
    want = gdn.residual_norm_backward(c.dh, c.dn, c.x, c.y, **c.args())
    ws, whole = _workspace(size)
    got = gdn.residual_norm_backward(c.dh, c.dn, c.x, c.y, **c.args(), workspace=ws)
    torch.cuda.synchronize()
    assert (whole[:G] == 0x5A).all() and (whole[-G:] == 0x5A).all() and not (ws == 255).all()
    for a, b in zip(got, want):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))


REACH = [
    # kind, form, page, width (positions: page * width), window, sinks
    ("bf16", "bf16", 16, 5, 0, 0),          # 80 positions: not cut
    ("bf16", "bf16", 16, 5, 33, 7),
    ("f32", "f32", 64, 20, 0, 0),           # 1280: cut
    ("f32", "f32", 64, 20, 700, 40),
    ("bf16", "mxfp8", 32, 100, 0, 0),
    ("f32", "mxfp4", 16, 70, 900, 1),
]


@pytest.mark.parametrize("kind,form,page,width,window,sinks", REACH)
def test_attention_of_lengths_beyond_a_full_table(kind, form, page, width, window, sinks):
    """Every page of the table is there; lengths behind its end count as its end, and so does a window's."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    reach = page * width
    full = [reach] * 5
    q, cache, table, kv, vv = _attention_case(kind, form, full, 4, 2, 64, page, window, sinks, 41)
    given = [reach, reach + 1, reach + 1000, 2 ** 31 - 1, reach - 1]
    assert (table >= 0).all() and table.shape == (5, width)
    lse = torch.empty((5, 4), device="cuda")
    y = gdn.attention_step(q, cache, i32(table), i32(given), window=window, sinks=sinks, lse=lse)
    # (of the last sequence one token more is hidden, and with a window another one seen: garbage there, so its own case)
    want = _expect(q[:4], table[:4], full[:4], kv, vv, 0.125, window, sinks, kind)
    _check_attention(y[:4], lse[:4], want, kind)
    if not window:
        _check_attention(y[4:], lse[4:], _expect(q[4:], table[4:], given[4:], kv, vv, 0.125, 0, 0, kind), kind)


def test_offsets_that_do_not_start_at_zero():
    """Rows in front of the first sequence are of no sequence: not written to the cache, not read into, not normed, and
    in no sum."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    T, H, d, page, first = 330, 2, 64, 16, 200
    off, table, start = i32([first, 240, 320]), i32([list(range(20)), list(range(20, 40))]), i32([250, 5])
    k, v = randn(1, T, H, d), randn(2, T, H, d)
    cache, want = gdn.kv_cache(40, H, page, d), gdn.kv_cache(40, H, page, d)
    gdn.kv_write(k, v, cache, table, start, seq_offsets=off)
    gdn.kv_write(k[first:].contiguous(), v[first:].contiguous(), want, table, start, seq_offsets=off - first)
    assert torch.equal(cache.k, want.k) and torch.equal(cache.v, want.v)
    ko, vo = torch.full_like(k, 7), torch.full_like(v, 7)
    gdn.kv_read(cache, table, T, start, seq_offsets=off, k_out=ko, v_out=vo)
    assert (ko[:first] == 7).all() and torch.equal(ko[first:320], k[first:320]) and torch.equal(vo[first:320], v[first:320])
    D = 136
    x, y, dh, dn = (randn(s, T, D) for s in range(4))
    w, gate = torch.linspace(0.5, 1.5, D, device="cuda"), torch.randn(2, D, device="cuda")
    args = dict(gate=gate, weight=w, post_weight=w)
    h, nn = torch.full_like(x, 7), torch.full_like(x, 7)
    gdn.residual_norm(x, y, **args, seq_offsets=off, out=h, norm_out=nn)
    cut = [t[first:].contiguous() for t in (x, y, dh, dn)]
    eh, en = gdn.residual_norm(*cut[:2], **args, seq_offsets=off - first)
    assert (h[:first] == 7).all() and (nn[:first] == 7).all()
    assert torch.equal(h[first:320], eh[:120]) and torch.equal(nn[first:320], en[:120])
    got = gdn.residual_norm_backward(dh, dn, x, y, **args, seq_offsets=off)
    want = gdn.residual_norm_backward(*cut[2:], *cut[:2], **args, seq_offsets=off - first)
    assert torch.equal(got[0][first:320], want[0][:120]) and torch.equal(got[1][first:320], want[1][:120])
    for g, e in zip(got[2:], want[2:]):  # (sums over 120 rows in two orders)
        assert torch.allclose(g, e, rtol=0, atol=240 * U * 120 * 64)
