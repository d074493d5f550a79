"""Sizes of the layer operators at the ends of what a launch can count, on the host."""
import pytest

import gated_delta_rule_scan_amd as gdn
from test_layer_abi import HIP, UNSUPPORTED, no_gpu, ssm


def _scan(B, T, D, N, **more):
    """B sequences of T tokens in one buffer each, one group, without states (2^34 bytes lie between the buffers)."""
    rows = {f"{r}_stride_{k}": (D if k == "t" else T * D) for r in ("x", "dt", "z", "out") for k in "tb"}
    rows.update({f"{r}_stride_{k}": (N if k == "t" else T * N) for r in "bc" for k in "tb"})
    assert B * T * max(D, N) * 2 <= 1 << 34
    return ssm(**dict(dict(B=B, T=T, D=D, N=N, G=1, state_in=None, state_out=None, slots=0), **rows, **more))


@no_gpu
@pytest.mark.parametrize("B,T,D,N", [(65537, 16, 4096, 16), (65536, 1, 16384, 16), (1 << 20, 4, 1024, 16), (1 << 22, 4, 64, 256)])
def test_unsplit_scans_need_no_carry(B, T, D, N):
    """B D N of 2^32 and more: the kernel that carries states between chunks could not be launched, and is not."""
    assert B * D * N >= 1 << 32
    p = gdn.gdn_ssm_problem_t(B=B, T=T, D=D, N=N, G=1, dtype=gdn.GDN_DTYPE_BF16)
    assert gdn.gdn_ssm_workspace_bytes(p) == 0
    assert _scan(B, T, D, N) == HIP


def test_grids_beyond_the_launch_are_refused():
    """The scan's own grid passes 2^32 work items."""
    assert _scan(1 << 25, 1, 64, 1) == UNSUPPORTED


@pytest.mark.gpu
def test_many_sequences_and_channels():
    """One call of 65537 sequences equals the calls of its halves."""
    import torch

    B, T, D, N = 65537, 2, 4096, 16
    torch.manual_seed(71)
    x, dt = (torch.randn(B, T, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    A, b, c = -torch.rand(D, N, device="cuda"), *(torch.randn(B, T, N, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    call = lambda s: gdn.selective_scan(x[s], dt[s], A, b[s], c[s], want_state=False)[0]
    y = call(slice(None))
    for s in (slice(0, 32768), slice(32768, B)):
        assert torch.equal(y[s], call(s))
