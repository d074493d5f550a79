"""Workspaces of the attention step and the seam's gradients on the host: which calls need one, and which are refused
for it."""
import os

import pytest

import gated_delta_rule_scan_amd as gdn
from test_hybrid_abi import attention, norm_problem
from test_layer_abi import HIP, INVALID, addr


def size(**over):
    f = dict(B=2, Hq=8, Hk=4, d=128, pages=100, page=16, table_width=1000, dtype=1, format=1)
    return gdn.gdn_attention_workspace_bytes(gdn.gdn_attention_problem_t(**{**f, **over}))


def test_attention_of_thousands_of_sequences_is_not_cut():
    """(Each workgroup of a cut call goes through all lengths.)"""
    assert size(B=1000) > 0
    assert all(size(B=B, Hk=Hk) == 0 for B in (1024, 5000, 1 << 20) for Hk in (1, 8))


LONG = dict(table_width=1000, window=0, workspace=addr(20))


def test_attention_workspace_is_as_large_as_it_says():
    need = size(format=1)
    assert need > 0 and need % 256 == 0
    assert attention(**LONG, workspace_bytes=need - 1) == gdn.GDN_ERR_WORKSPACE_TOO_SMALL
    assert attention(**LONG, workspace_bytes=0) == gdn.GDN_ERR_WORKSPACE_TOO_SMALL
    if not os.path.exists("/dev/kfd"):
        assert attention(**LONG, workspace_bytes=need) == HIP
        assert attention(workspace=None, workspace_bytes=0) == HIP  # 80 positions: none needed


@pytest.mark.parametrize("at", [None, addr(20) + 64, addr(20) + 128, addr(0), addr(1), addr(2) + (100 << 14) - 256, addr(3), addr(6),
                                addr(7), addr(8), addr(1) - 512])
def test_attention_workspaces_that_are_refused(at):
    """Missing, misaligned, over q, out, either pool, the table, the lengths, lse; ending in out."""
    assert attention(**{**LONG, "workspace": at, "workspace_bytes": size(format=1)}) == INVALID


@pytest.mark.parametrize("form", [2, 3])
@pytest.mark.parametrize("pool", [4, 5])
def test_attention_workspaces_over_scales_are_refused(form, pool):
    assert attention(**{**LONG, "format": form, "workspace": addr(pool), "workspace_bytes": size(format=form)}) == INVALID


def test_norm_workspaces_of_every_form():
    """As many partial rows for each gradient, whichever they are."""
    one = gdn.gdn_norm_workspace_bytes(norm_problem(gate=None, post_weight=None))
    assert one > 0
    for given in range(8):
        over = {k: None for i, k in enumerate(("gate", "post_weight", "weight")) if not given >> i & 1}
        assert gdn.gdn_norm_workspace_bytes(norm_problem(**over)) == bin(given).count("1") * one
