"""The cache, the attention step and the seam as they run together and in a
program's surroundings: a hybrid model's softmax layer over a prompt and single
tokens, a window of the cache into the token scan; graph capture and replay;
other streams, beside pending work; guarded and poisoned buffers; offsets beyond
32 bits; torch.compile; refusals."""
import numpy as np
import pytest

import hybrid_oracle as oracle
from layer_oracle import check
from test_gpu_hybrid import SeamCase, i32
from test_gpu_layer import Rng, n, offsets
from test_gpu_layer_together import G, _clone, _guarded

pytestmark = pytest.mark.gpu

LONG = 20_000_000  # cycles of waiting on the device, some ten milliseconds


class Stream:
    """A softmax layer's pages: taken from a pool as sequences grow."""

    def __init__(self, pages, page, width, B):
        self.free, self.page = list(np.random.default_rng(1).permutation(pages)), page
        self.table = np.full((B, width), -1, np.int32)
        self.lens = [0] * B

    def grow(self, b, tokens):
        for p in range(-(-self.lens[b] // self.page), -(-(self.lens[b] + tokens) // self.page)):
            self.table[b, p] = self.free.pop()
        self.lens[b] += tokens


@pytest.mark.parametrize("kind,form", [("bf16", "bfloat16"), ("f32", "float32"), ("bf16", "mxfp8"), ("f32", "mxfp4")])
def test_softmax_layer_prompt_then_tokens(kind, form):
    """Seam -> projections -> rotary -> cache -> attention -> seam: prompts of different lengths packed, then tokens one
    by one.  Every attention is checked against the keys and values that the layer has computed so far."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    r = Rng(71)
    lens, B, Hq, Hk, d, D, page = [37, 1, 70], 3, 4, 2, 64, 128, 16
    W = [r.t(D, m * d, kind=kind, scale=D ** -0.5) for m in (Hq, Hk, Hk)]
    Wo = r.t(Hq * d, D, kind=kind, scale=0.1)
    nw, pw, gate = r.t(D, mean=1.0, scale=0.1), r.t(D, mean=1.0, scale=0.1), r.t(B, D, mean=0.5, scale=0.2)
    f = gdn.rotary_frequencies(d)[0].cuda()
    cache, pages = gdn.kv_cache(40, Hk, page, d, form), Stream(40, page, 8, B)
    seen = [[] for _ in range(B)]  # (k, v) rows as the layer wrote them
    heads = lambda x, w, m: (x @ w).unflatten(-1, (m, d))
    off = offsets(lens)
    x = r.t(sum(lens), D, kind=kind)
    _, norm = gdn.residual_norm(x, weight=nw)
    pos = torch.cat([torch.arange(m, device="cuda") for m in lens])
    q, k = gdn.rotary(heads(norm, W[0], Hq)[None], heads(norm, W[1], Hk)[None], f, pos[None])
    k, v = k[0], heads(norm, W[2], Hk)
    for b, m in enumerate(lens):
        pages.grow(b, m)
    gdn.kv_write(k, v, cache, i32(pages.table), seq_offsets=off)
    for b in range(B):
        lo, hi = sum(lens[:b]), sum(lens[: b + 1])
        seen[b] = [(n(k)[t], n(v)[t]) for t in range(lo, hi)]
    held = (lambda a: oracle.decode(*oracle.encode(a, form), form)) if form.startswith("mx") else (lambda a: a)
    x, y, norm = r.t(B, D, kind=kind), None, None
    for step in range(20):
        start = i32(pages.lens)
        for b in range(B):
            pages.grow(b, 1)
        h, norm = gdn.residual_norm(x, y, gate=gate if y is not None else None, post_weight=pw if y is not None else None,
                                    weight=nw)
        q, k = gdn.rotary(heads(norm, W[0], Hq)[:, None], heads(norm, W[1], Hk)[:, None], f, start[:, None])
        v = heads(norm, W[2], Hk)
        table = i32(pages.table)
        gdn.kv_write(k[:, 0], v, cache, table, start)
        lse = torch.empty((B, Hq), device="cuda")
        o = gdn.attention_step(q[:, 0], cache, table, i32(pages.lens), lse=lse)
        for b in range(B):
            seen[b].append((n(k)[b, 0], n(v)[b]))
            kk, vv = held(np.stack([s[0] for s in seen[b]])), held(np.stack([s[1] for s in seen[b]]))
            for kh in range(Hk):
                g = slice(2 * kh, 2 * kh + 2)
                (e, eb), (l, lb) = oracle.attend(n(q)[b, 0, g], kk[:, kh], vv[:, kh], d ** -0.5, kind == "bf16")
                check(n(o)[b, g], e, eb, kind, f"token {step}")
                check(n(lse)[b, g], l, lb, "f32", f"token {step}")
        x, y = h, o.flatten(1) @ Wo
    # the whole cache comes back as it was written
    gk, gv = gdn.kv_read(cache, i32(pages.table), sum(pages.lens), seq_offsets=offsets(pages.lens), dtype=x.dtype)
    want = [held(np.stack([s[i] for b in range(B) for s in seen[b]])) for i in (0, 1)]
    assert np.array_equal(n(gk), want[0]) and np.array_equal(n(gv), want[1])


def test_window_of_the_cache_into_the_token_scan():
    """Keys and values of a window, read back, fold into a recurrent state: the scan of the original rows, bit for bit."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    r = Rng(72)
    B, T, H, d, page = 2, 300, 3, 64, 32
    q, k, v = (r.t(B, T, H, d, kind="bf16") for _ in range(3))
    la, beta = -r.t(1, B, 200, H).abs() * 0.1, torch.sigmoid(r.t(1, B, 200, H))
    cache = gdn.kv_cache(2 * 10 + 1, H, page, d)
    table = i32(np.random.default_rng(3).permutation(20).reshape(2, 10))
    gdn.kv_write(k, v, cache, table)
    start = i32([100, 57])
    gk, gv = gdn.kv_read(cache, table, 200, start)
    wk, wv = (torch.stack([t[0, 100:300], t[1, 57:257]]) for t in (k, v))
    want = gdn.forward(q[:, :200].contiguous(), wk, wv, la, beta)
    got = gdn.forward(q[:, :200].contiguous(), gk, gv, la, beta)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_attention_beside_the_recurrent_step():
    """A hybrid model's token: three recurrent blocks' steps and one softmax block on one stream, slots and pages of the
    same sequences; two runs give the same bits."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    def run():
        r = Rng(73)
        B, H, d, D = 4, 2, 64, 128
        pool, slots = r.t(6, H, d, d, scale=0.1), i32([5, 0, 3, 1])
        cache, table = gdn.kv_cache(30, H, 16, d, "mxfp8"), i32(np.arange(24).reshape(4, 6))
        nw = r.t(D, mean=1.0, scale=0.1)
        x = r.t(B, D, kind="bf16")
        outs = []
        for t in range(6):
            y = None
            for block in range(4):
                x, u = gdn.residual_norm(x, y, weight=nw, residual_scale=1.0)
                q, k, v = ((u * s).unflatten(-1, (H, d)).contiguous() for s in (1.0, 0.5, 2.0))
                if block < 3:
                    o = gdn.delta_step(q, k, v, -torch.ones(B, H, device="cuda") * 0.1, torch.full((B, H), 0.5, device="cuda"),
                                       pool, slots)
                else:
                    at = torch.full((B,), t, dtype=torch.int32, device="cuda")
                    gdn.kv_write(k, v, cache, table, at)
                    o = gdn.attention_step(q, cache, table, at + 1)
                y = o.flatten(1).to(torch.bfloat16)
            outs.append(x.clone())
        return torch.stack(outs)

    a, b = run(), run()
    assert torch.equal(a, b) and torch.isfinite(a).all()


# ---- in a program's surroundings ----

def _all_calls(r, kind="bf16"):
    """name -> (function of fresh static inputs, those inputs): outputs and pools returned."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    B, Hq, Hk, d, page = 3, 6, 2, 64, 16
    lens = [700, 0, 130]
    used = [-(-x // page) for x in lens]
    table = np.full((B, 60), -1, np.int32)
    order = np.random.default_rng(5).permutation(sum(used))
    for b in range(B):
        table[b, : used[b]] = order[sum(used[:b]): sum(used[: b + 1])]
    table, lengths, off = i32(table), i32(lens), offsets(lens)
    pools = [r.t(sum(used) + 2, Hk, page, d, kind=kind) for _ in range(2)]
    q = r.t(B, Hq, d, kind=kind)
    k, v = r.t(sum(lens) + 3, Hk, d, kind=kind), r.t(sum(lens) + 3, Hk, d, kind=kind)
    form = "mxfp8"

    def write(k, v, p0, p1, **o):
        gdn.kv_write(k, v, (p0, p1), table, seq_offsets=off, **o)
        return p0, p1

    def write8(k, v, p0, p1, s0, s1, **o):
        gdn.kv_write(k, v, (p0.view(torch.float8_e4m3fn), p1.view(torch.float8_e4m3fn), s0, s1), table, seq_offsets=off, **o)
        return p0, p1, s0, s1

    def attend(q, p0, p1, **o):
        lse = torch.zeros((B, Hq), device="cuda")
        return gdn.attention_step(q, (p0, p1), table, lengths, lse=lse, **o), lse

    c8 = gdn.kv_cache(sum(used) + 2, Hk, page, d, form)
    c = SeamCase(kind, [700, 0, 130], 136, True, "sequence", True, True, 0.9, "plain")
    args = c.args()
    back = lambda dh, dn, x, y, **o: [t for t in gdn.residual_norm_backward(dh, dn, x, y, **args, **o) if t is not None]
    return {
        "write": (write, dict(k=k, v=v, p0=pools[0], p1=pools[1])),
        "write 8 bits": (write8, dict(k=k, v=v, p0=c8.k.view(torch.uint8), p1=c8.v.view(torch.uint8), s0=c8.k_scales, s1=c8.v_scales)),
        "read": (lambda p0, p1, **o: gdn.kv_read((p0, p1), table, sum(lens) + 3, seq_offsets=off, **o), dict(p0=pools[0], p1=pools[1])),
        "attention": (attend, dict(q=q, p0=pools[0], p1=pools[1])),
        "attention, short": (lambda q, p0, p1, **o: (gdn.attention_step(q, (p0, p1), table[:, :20].contiguous(), lengths, **o),),
                             dict(q=q, p0=pools[0], p1=pools[1])),
        "seam": (lambda x, y, **o: gdn.residual_norm(x, y, **args, **o), dict(x=c.x, y=c.y)),
        "seam backward": (back, dict(dh=c.dh, dn=c.dn, x=c.x, y=c.y)),
    }


NAMES = ["write", "write 8 bits", "read", "attention", "attention, short", "seam", "seam backward"]


@pytest.mark.parametrize("name", NAMES)
def test_capture_and_replay(name):
    """Captured once, replayed three times on new inputs with eager work between: every replay equals an eager call bit
    for bit."""
    import torch

    r = Rng(74)
    fn, kw = _all_calls(r)[name]
    vary = [k for k in ("q", "k", "v", "x", "y", "dn") if k in kw] or ["p0", "p1"]
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
        want = [w.clone() for w in fn(**{**_clone(kw), **{k: v.clone() for k, v in new.items()}})]
        torch.randn(1000, 1000, device="cuda").sum()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), f"replay {i}"


@pytest.mark.parametrize("name", NAMES)
def test_repeats_and_other_streams_are_bitwise_equal(name):
    import torch

    fn, kw = _all_calls(Rng(75))[name]
    first = [t.clone() for t in fn(**_clone(kw))]
    for a, b in zip(first, fn(**_clone(kw))):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    for _ in range(3):
        own = _clone(kw)
        side.wait_stream(torch.cuda.current_stream())
        if name.startswith("attention"):
            with torch.cuda.stream(side):  # (the test's own tensors of the call, too)
                got = fn(**own)
        else:
            got = fn(**own, stream=side)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(first, got):
            assert torch.equal(a, b)
        del junk, got, own


@pytest.mark.parametrize("name", NAMES)
def test_two_calls_at_once(name):
    """The same call on two streams at the same time, each with outputs and workspace of its own."""
    import torch

    fn, kw = _all_calls(Rng(76))[name]
    want = [t.clone() for t in fn(**_clone(kw))]
    sides = [torch.cuda.Stream() for _ in range(2)]
    own = [_clone(kw) for _ in sides]
    torch.cuda.synchronize()
    got = [[] for _ in sides]
    for _ in range(5):
        for i, s in enumerate(sides):
            with torch.cuda.stream(s):
                got[i].append(fn(**own[i]))
    torch.cuda.synchronize()
    for outs in got:
        for o in outs:
            for a, b in zip(o, want):
                assert torch.equal(a, b)


def test_results_share_no_memory_with_pending_work():
    """Blocks of the very sizes that a call allocates are freed on the current stream while a fill of them is still to
    come there; the call runs on another stream."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    calls = _all_calls(Rng(77), "f32")
    _, a = calls["attention"]
    p = gdn.gdn_attention_problem_t(B=3, Hq=6, Hk=2, d=64, pages=a["p0"].shape[0], page=16, table_width=60, dtype=0, format=0,
                                    window=0, sinks=0)
    ws = gdn.gdn_attention_workspace_bytes(p)
    assert ws
    c = SeamCase("f32", [700, 0, 130], 136, True, "sequence", True, True, 0.9, "plain")
    np_ = gdn.gdn_norm_problem_t(B=3, T=832, D=136, gate_stride_b=136, dtype=0, residual_scale=1.0, eps=1e-6)
    np_.gate = np_.post_weight = np_.weight = np_.seq_offsets = 1 << 20
    nws = gdn.gdn_norm_workspace_bytes(np_)
    assert nws
    rows = c.x.numel() * 4
    sizes = {"read": [833 * 2 * 64 * 4], "attention": [3 * 6 * 64 * 4, ws], "seam": [rows], "seam backward": [rows, nws, 3 * 136 * 4, 136 * 4]}
    for name, sz in sizes.items():
        fn, kw = calls[name]
        want = [t.clone() for t in fn(**kw)]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        if name == "attention":
            lse = torch.zeros((3, 6), device="cuda")
        torch.cuda._sleep(LONG)
        late = [torch.empty(m, dtype=torch.uint8, device="cuda").fill_(255) for m in sz for _ in range(3)]
        taken = {t.data_ptr() for t in late}
        del late
        got = fn(**kw, stream=side)
        assert name == "attention" or not taken & {t.data_ptr() for t in got}
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            if name != "attention" or i == 0:  # (the test's lse is the current stream's)
                assert torch.equal(x, y), name


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("name", NAMES)
def test_guard_zones_and_poisoned_outputs(name, kind):
    """Every buffer sits between guard zones that stay intact; inputs keep their values; poisoned outputs are written
    everywhere but in rows of no sequence."""
    import torch

    fn, kw = _all_calls(Rng(78), kind)[name]
    want = [t.clone() for t in fn(**_clone(kw))]
    wholes, own = [], {}
    for k, v in kw.items():
        own[k], whole = _guarded(v)
        wholes.append(whole)
    given = {"read": ("k_out", "v_out"), "seam": ("out", "norm_out"), "seam backward": ("dx", "dy"), "attention": ("out",),
             "attention, short": ("out",)}.get(name, ())
    outs = {}
    for i, k in enumerate(given):
        outs[k], whole = _guarded(torch.full_like(want[i], float("nan")))
        wholes.append(whole)
    if name.startswith("attention"):
        ws, whole = _guarded(torch.zeros(1 << 22, dtype=torch.uint8, device="cuda"))
        outs["workspace"] = ws
        wholes.append(whole)
    if name == "seam backward":
        outs["workspace"], whole = _guarded(torch.zeros(1 << 24, dtype=torch.uint8, device="cuda"))
        wholes.append(whole)
    got = fn(**own, **outs)
    torch.cuda.synchronize()
    for whole in wholes:
        assert (whole[:G] == 0x5A).all() and (whole[-G:] == 0x5A).all()
    rows = 830  # of sequences, in packed outputs
    for i, (a, b) in enumerate(zip(got, want)):
        packed = i < len(given) and not name.startswith("attention")
        assert torch.equal(a[:rows], b[:rows]) if packed else torch.equal(a, b)
        assert not packed or torch.isnan(a[rows:]).all()
    written = {"write": ("p0", "p1"), "write 8 bits": ("p0", "p1", "s0", "s1")}.get(name, ())
    for k, v in kw.items():
        assert k in written or torch.equal(own[k], v), k


def test_offsets_beyond_32_bits():
    """Rows more than 2^32 bytes apart: sequences at the ends of one 9 GB buffer."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    r = Rng(79)
    T, H, d, D = 40, 2, 64, 128
    buf = torch.zeros((1 << 32) + (1 << 29), dtype=torch.bfloat16, device="cuda")
    far = 1 << 32  # elements
    view = lambda at, *s: torch.as_strided(buf, (2, T, *s), (far, D, *([d] * (len(s) - 1)), 1), at)
    small = r.t(2, T, H, d, kind="bf16")
    k, v = view(0, H, d), view(1 << 20, H, d)
    k.copy_(small)
    v.copy_(small * 2)
    caches = [gdn.kv_cache(7, H, 16, d, "mxfp8") for _ in range(2)]
    table = i32([[0, 1, 2], [3, 4, 5]])
    gdn.kv_write(k, v, caches[0], table)
    gdn.kv_write(small, small * 2, caches[1], table)
    for a, b in zip(*caches):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    ko, vo = view(1 << 21, H, d), view(1 << 22, H, d)
    gdn.kv_read(caches[0], table, T, k_out=ko, v_out=vo)
    want = gdn.kv_read(caches[1], table, T)
    assert torch.equal(ko, want[0]) and torch.equal(vo, want[1])
    x, y, h, nn = (view(at, D) for at in (0, 1 << 20, 1 << 23, 1 << 24))
    w = r.t(D, mean=1.0)
    xs, ys = x.contiguous(), y.contiguous()
    want = gdn.residual_norm(xs, ys, post_weight=w, weight=w)
    gdn.residual_norm(x, y, post_weight=w, weight=w, out=h, norm_out=nn)
    assert torch.equal(h, want[0]) and torch.equal(nn, want[1])
    want = gdn.residual_norm_backward(xs, ys, xs, ys, post_weight=w, weight=w)
    got = gdn.residual_norm_backward(x, y, x, y, post_weight=w, weight=w, dx=h, dy=nn)
    for a, b in zip(got, want):
        assert a is b is None or torch.equal(a, b)
    qs = r.t(2, H, d, kind="bf16")
    q, o = (torch.as_strided(buf, (2, H, d), (far, d, 1), at) for at in (1 << 25, 1 << 26))
    q.copy_(qs)
    lens = i32([40, 33])
    want = gdn.attention_step(qs, caches[0], table, lens)
    gdn.attention_step(q, caches[0], table, lens, out=o)
    assert torch.equal(o, want)


def test_compiled_calls_equal_eager():
    import torch

    import gated_delta_rule_scan_amd as gdn

    gdn.register_torch_ops()
    r = Rng(80)
    H, d, D = 2, 64, 128
    cache = gdn.kv_cache(9, H, 16, d, "mxfp8")
    table, w, gate = i32([[0, 4, 2], [7, 1, 3]]), r.t(D, mean=1.0), r.t(2, D)
    x, y, dh, dn = (r.t(2, 30, D, kind="bf16") for _ in range(4))

    def fn(x, y, k, v, ks, vs):
        h, m = torch.ops.gdn.residual_norm(x, y, gate, w, w, 1.0, 1e-6, None)
        rows = m.unflatten(-1, (H, d))
        torch.ops.gdn.kv_write(rows, rows, k, v, ks, vs, table, None, None)
        o, lse = torch.ops.gdn.attention_step(rows[:, -1], k, v, ks, vs, table, torch.full((2,), 30, dtype=torch.int32, device="cuda"),
                                              None, 0, 0)
        a, b = torch.ops.gdn.kv_read(k, v, ks, vs, table, 30, None, None, torch.bfloat16)
        g = torch.ops.gdn.residual_norm_backward(dh, dn, x, y, gate, w, w, 1.0, 1e-6, None)
        return h, o * 2, lse, a, b, *g

    c1, c2 = [t.clone() for t in cache], [t.clone() for t in cache]
    got = torch.compile(fn, backend="aot_eager", fullgraph=True)(x, y, *c1)
    want = fn(x, y, *c2)
    for a, b in zip(got + tuple(c1), want + tuple(c2)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_refusals():
    """What the binding refuses before any launch: shapes, types, devices, memory that would meet."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    z = lambda *s, **k: torch.zeros(s, device="cuda", **k)
    t, l = z(2, 3, dtype=torch.int32), z(2, dtype=torch.int32)
    bf = dict(dtype=torch.bfloat16)
    pool, c8, c4 = (z(5, 2, 16, 64, **bf), z(5, 2, 16, 64, **bf)), gdn.kv_cache(5, 2, 16, 64, "mxfp8"), gdn.kv_cache(5, 2, 16, 64, "mxfp4")
    q, k = z(2, 4, 64, **bf), z(2, 7, 2, 64, **bf)
    ok = gdn.attention_step(q, pool, t, l)
    assert ok.shape == q.shape
    for bad in (lambda: gdn.attention_step(z(2, 3, 64, **bf), pool, t, l),            # heads
                lambda: gdn.attention_step(z(2, 4, 128, **bf), pool, t, l),           # channels
                lambda: gdn.attention_step(q.float(), pool, t, l),                    # the cache's type
                lambda: gdn.attention_step(q, pool, t[:1], l), lambda: gdn.attention_step(q, pool, t.long(), l),
                lambda: gdn.attention_step(q, pool, t, l.long()), lambda: gdn.attention_step(q, pool, t.cpu(), l),
                lambda: gdn.attention_step(q, pool, t, l, window=-1), lambda: gdn.attention_step(q, pool, t, l, lse=z(2, 3)),
                lambda: gdn.attention_step(q, pool, t, l, out=z(2, 4, 64)),
                lambda: gdn.attention_step(q, (pool[0], pool[1][:4]), t, l),
                lambda: gdn.attention_step(q, (c8.k, c8.v, c8.k_scales, c8.v_scales[:, :, :, :1]), t, l),
                lambda: gdn.attention_step(q, (c8.k, c8.v, c8.k_scales, None), t, l),
                lambda: gdn.attention_step(q, pool, t, l, workspace=z(100)),
                lambda: gdn.kv_write(z(2, 7, 3, 64, **bf), z(2, 7, 3, 64, **bf), pool, t),
                lambda: gdn.kv_write(k, k[:, :6], pool, t), lambda: gdn.kv_write(k.float(), k.float(), pool, t),
                lambda: gdn.kv_write(k, k, pool, t, start=z(3, dtype=torch.int32)),
                lambda: gdn.kv_write(k.transpose(2, 3), k.transpose(2, 3), pool, t),
                lambda: gdn.kv_write(k, k, pool, t, seq_offsets=z(3, dtype=torch.int32)),
                lambda: gdn.kv_read(pool, t, -1), lambda: gdn.kv_read(pool, t, 5, dtype=torch.float32),
                lambda: gdn.kv_read(pool, t, 5, k_out=z(2, 5, 2, 64, **bf)),
                lambda: gdn.kv_read(pool, t, 5, k_out=z(2, 4, 2, 64, **bf), v_out=z(2, 4, 2, 64, **bf))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: gdn.attention_step(q, pool[0], t, l), lambda: gdn.attention_step(q, (pool[0].half(), pool[1].half()), t, l),
                lambda: gdn.attention_step(q, (c8.k, c8.v), t, l), lambda: gdn.attention_step(q, pool, t, l, window="x"),
                lambda: gdn.attention_step(q, pool, t, l, scale="x"), lambda: gdn.kv_read(c4, t, 2.5)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(gdn.GdnError):  # over the cache
        gdn.kv_read(pool, t, 16, k_out=pool[0].view(-1)[: 2 * 16 * 2 * 64].view(2, 16, 2, 64), v_out=z(2, 16, 2, 64, **bf))
    with pytest.raises(gdn.GdnError):
        gdn.attention_step(q, pool, t, l, scale=float("inf"))
    with pytest.raises(gdn.GdnError):
        gdn.attention_step(z(2, 4, 32, **bf), (z(5, 2, 16, 32, **bf), z(5, 2, 16, 32, **bf)), t, l)
    x, w = z(2, 5, 8), z(8)
    for bad in (lambda: gdn.residual_norm(x), lambda: gdn.residual_norm(x, gate=w, weight=w), lambda: gdn.residual_norm(x, x, weight=z(7)),
                lambda: gdn.residual_norm(x, x, gate=z(3, 8), weight=w), lambda: gdn.residual_norm(x, z(2, 5, 7), weight=w),
                lambda: gdn.residual_norm(x, x, norm_out=x), lambda: gdn.residual_norm(x, x.bfloat16(), weight=w),
                lambda: gdn.residual_norm(x[0], x[0], weight=w, seq_offsets=z(2, dtype=torch.int32), out=z(5, 8)),
                lambda: gdn.residual_norm_backward(None, None, x, x), lambda: gdn.residual_norm_backward(x, x, x, x),
                lambda: gdn.residual_norm_backward(x, None, x, x, weight=w), lambda: gdn.residual_norm_backward(x, None, x, dy=x),
                lambda: gdn.residual_norm(z(2, 5, 8, 1), weight=w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gdn.GdnError):
        gdn.residual_norm(x, x, weight=w, eps=-1.0)
    with pytest.raises(gdn.GdnError):  # n over the residual stream
        gdn.residual_norm(x, z(2, 5, 8), weight=w, norm_out=x)
