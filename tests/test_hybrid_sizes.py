"""Workspaces of the attention step on the host: which calls need one, and which are refused for it."""
import pytest

import gated_delta_rule_scan_amd as gdn
from test_hybrid_abi import attention


def size(**over):
    f = dict(B=2, Hq=8, Hk=4, d=128, pages=100, page=16, table_width=1000, dtype=1, format=1)
    return gdn.gdn_attention_workspace_bytes(gdn.gdn_attention_problem_t(**{**f, **over}))


def test_attention_of_thousands_of_sequences_is_not_cut():
    """(Each workgroup of a cut call goes through all lengths.)"""
    assert size(B=1000) > 0
    assert all(size(B=B, Hk=Hk) == 0 for B in (1024, 5000, 1 << 20) for Hk in (1, 8))
