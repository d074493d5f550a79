"""Options of the layer operators' C calls, on the host."""
import pytest

import gated_delta_rule_scan_amd as gdn
from test_layer_abi import HIP, INVALID, addr, conv, no_gpu, ssm, step

ZERO = gdn.GDN_LAYER_OPT_ZERO_UNUSED
CALLS = {"conv": conv, "conv step": lambda **k: conv(step=True, **k), "ssm": ssm, "ssm step": lambda **k: ssm(step=True, **k),
         "step": step}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("options", [512, ZERO | 512, -1])
def test_unknown_options_are_refused(name, options):
    assert CALLS[name](options=options) == INVALID


def test_rotary_has_no_unused_rows():
    from test_layer_abi import rotary

    assert rotary(options=ZERO) == INVALID


@no_gpu
@pytest.mark.parametrize("name", CALLS)
def test_zeroing_reaches_the_launch(name):
    assert CALLS[name](options=ZERO) == HIP
    if name in ("conv", "ssm"):
        assert CALLS[name](options=ZERO, seq_offsets=addr(11)) == HIP
    assert CALLS[name](options=ZERO, state_index=addr(11), slots=5) == HIP


@no_gpu
def test_zeroing_goes_with_the_other_options():
    assert ssm(options=ZERO | gdn.GDN_SSM_OPT_SOFTPLUS) == HIP
    assert step(options=ZERO | gdn.GDN_OPT_NO_ERASE | gdn.GDN_OPT_EXCLUSIVE_FORWARD) == HIP
