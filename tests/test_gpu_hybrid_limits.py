"""The largest batches of the cache, its attention and the seam on the GPU: more workgroups than one launch takes,
against the same rows in calls that need fewer; more sequences than are cut."""
import pytest

from layer_oracle import U
from test_gpu_hybrid import _attention_case, _check_attention, _expect, i32
from test_gpu_layer import _torch

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
def test_attention_of_a_thousand_sequences_in_a_wide_table(kind, form):
    """Not cut, short ones and one long one."""
    import gated_delta_rule_scan_amd as gdn

    torch = _torch()
    lens = [3, 40, 0, 17] * 256 + [4100, 700]
    q, cache, table, kv, vv = _attention_case(kind, form, lens, 4, 2, 64, 64, 0, 0, 31, width=100)
    lse = torch.empty((len(lens), 4), device="cuda")
    y = gdn.attention_step(q, cache, i32(table), i32(lens), lse=lse)
    _check_attention(y, lse, _expect(q, table, lens, kv, vv, 0.125, 0, 0, kind), kind)
