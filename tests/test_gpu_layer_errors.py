"""Errors of the layer operators' calls that come from torch itself keep their types."""
import pytest

pytestmark = pytest.mark.gpu


def test_out_of_memory_is_torchs():
    """An output that the allocator refuses (by a limit of its own: nothing is asked of the device) is torch's
    OutOfMemoryError, and the next call works."""
    import torch

    import gated_delta_rule_scan_amd as gdn

    x, w = torch.ones(1, 4, 64, device="cuda"), torch.ones(64, 4, device="cuda")
    wide = x[:, :1].expand(1 << 14, 1 << 12, 64)  # 16 GiB, of one row
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 30)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError) as e:
            gdn.causal_conv(wide, w)
        assert "frame #" not in str(e.value)  # no C++ trace
        y, _ = gdn.causal_conv(x, w, activation="none")
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert torch.equal(y[0, :, 0], torch.arange(1.0, 5.0, device="cuda"))
