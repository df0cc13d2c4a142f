"""Workspaces that callers hand to the native binding: no GPU needed."""
import pytest
import torch


def test_a_workspace_is_contiguous_memory_of_the_calls_device(fa_mod):
    """An expanded tensor says more bytes than it has; memory of the host or of
    another device is not the kernels' to write."""
    check = fa_mod.native().check_workspace
    with pytest.raises(ValueError, match="workspace must be on cuda:0, got cpu"):
        check(torch.empty(1 << 20, dtype=torch.uint8), 0)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        check(torch.empty(1, dtype=torch.uint8).expand(1 << 20), 0)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        check(torch.empty(64, 64, dtype=torch.uint8).t(), 0)
