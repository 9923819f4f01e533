"""Checks of the binding that need no GPU."""
import pytest
import torch

from entropy_active_span_gb300 import _ws_args


def test_workspace_arguments():
    """A workspace on another device than the tensors must not reach the kernels."""
    here = torch.device("cpu")
    assert _ws_args(torch.empty(40, dtype=torch.uint8), here)[1] == 40
    assert _ws_args(torch.empty(5, dtype=torch.int64), here)[1] == 40
    with pytest.raises(ValueError, match="ws is on cpu"):
        _ws_args(torch.empty(40, dtype=torch.uint8), torch.device("cuda", 0))
    with pytest.raises(ValueError, match="contiguous"):
        _ws_args(torch.empty(40, dtype=torch.uint8)[::2], here)
    with pytest.raises(TypeError):
        _ws_args(40, here)
