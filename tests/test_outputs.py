"""Outputs that the training operators allocate for a call: torch's own errors where there is no memory or no device."""

import pytest
import torch

from top_gating_expert_gb300 import _native as N
from top_gating_expert_gb300 import train


@pytest.mark.skipif(torch.cuda.is_available(), reason="there is a device")
def test_no_device(native_lib):
    """What torch.empty raises without a GPU, not a ValueError about the arguments."""
    with pytest.raises((RuntimeError, AssertionError)) as want:
        torch.empty(5, device="cuda")
    assert not issubclass(want.type, ValueError)
    with pytest.raises(RuntimeError):
        train._lists().outputs(0, N.MOE_F32, 0, 5)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [(1 << 44,), (4, 1 << 44)])
def test_no_memory(native_lib, rows):
    """64 TB are refused as torch refuses them (the allocator asks once and gets nothing); the next call works."""
    with pytest.raises(torch.OutOfMemoryError):
        train._lists().outputs(0, N.MOE_F32, 0, *rows)
    x, W = torch.ones(3, 8, device="cuda"), torch.ones(5, 8, device="cuda")
    loss, lse, stats = train.linear_cross_entropy(x, W, torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert stats[1].item() == 3
