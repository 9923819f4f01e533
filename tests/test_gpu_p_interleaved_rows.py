"""Logits and their gradient side by side in one buffer: what lies between their rows."""
import pytest
import torch

import entropy_active_span_gb300 as eas

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,V,pitch,at", [(5, 1000, 2000, 1000), (700, 129, 400, 150), (3, 40000, 80016, 40008)])
def test_gradient_between_the_rows(N, V, pitch, at, dtype):
    buf = torch.full((N, pitch), 7.0, dtype=dtype, device="cuda")
    x, d = buf[:, :V], buf[:, at:at + V]
    x.copy_(torch.randn(N, V, generator=torch.Generator().manual_seed(0)))
    dense = x.contiguous()
    t = torch.arange(N, dtype=torch.int32, device="cuda") % V
    lp, ent, lse, _, _ = eas.token_logprobs_fwd(dense, t)
    args = (torch.ones(N, device="cuda"), ent, dense, t, lse, ent)
    ref = eas.token_logprobs_bwd(*args)
    assert eas.token_logprobs_bwd(*args[:2], x, *args[3:], out=d) is d
    assert torch.equal(d, ref) and torch.equal(x, dense)
    assert (buf[:, V:at] == 7).all() and (buf[:, at + V:] == 7).all()
    # and the other way round
    d.copy_(dense)
    eas.token_logprobs_bwd(*args[:2], d, *args[3:], out=x)
    assert torch.equal(x, ref) and torch.equal(d, dense)
    with pytest.raises(eas.EasError, match="overlaps"):
        eas.token_logprobs_bwd(*args[:2], x, *args[3:], out=buf[:, V - 1:2 * V - 1])
