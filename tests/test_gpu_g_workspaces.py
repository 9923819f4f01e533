"""Workspaces that the operators around the LM head cannot write."""
import pytest
import torch

import entropy_active_span_gb300 as eas

pytestmark = pytest.mark.gpu


def calls():
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    w, ids = x[0].clone(), torch.zeros(4, dtype=torch.int32, device="cuda")
    return {
        "norm": (lambda ws: eas.rmsnorm_bwd(x, x, w, ws=ws), eas.rmsnorm_bwd_workspace_size(4, 64)),
        "lookup": (lambda ws: eas.embed_fwd(ids, x, ws=ws), 256),
        "gradient": (lambda ws: eas.embed_bwd(ids, x, 4, ws=ws), eas.embed_bwd_workspace_size(4, 64, 4)),
        "clip": (lambda ws: eas.clip_grad_norm([x], 1.0, ws=ws), eas.clip_grad_norm_workspace_size(1)),
    }


@pytest.mark.parametrize("name", ["norm", "lookup", "gradient", "clip"])
def test_workspaces(name):
    call, n = calls()[name]
    with pytest.raises(ValueError, match="ws is on cpu"):
        call(torch.empty(n, dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous"):
        call(torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2])
    with pytest.raises(TypeError):
        call(n)
    ws = torch.full((n // 8 + 1,), -1, dtype=torch.int64, device="cuda")     # any type: bytes count
    call(ws)
    assert eas.read_device_status(ws) == 0
