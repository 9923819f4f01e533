"""Scores of logits at scales far below 1, up to the least that fp32 has: every token is
as likely as any other, whatever a thread's last vectors hold.  Tolerances are those of
the other scales."""
import pytest
import torch

import entropy_active_span_gb300 as eas
from test_gpu_j_scores import check_bwd, check_fwd, make, make_tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1e-24, 1e-27, 1e-28, 1e-30, 1e-35, 1e-42])
# a CTA a row, a cluster a row, rows in turn by groups of four and of eight vectors, all with
# a last group that is not full
@pytest.mark.parametrize("N,V", [(400, 1000), (3, 9001), (330, 16401), (330, 26009), (320, 40003)])
def test_small_scales(N, V, scale, dtype):
    x = make(N, V, dtype, 3)
    tokens = make_tokens(N, V, 2)
    got = eas.token_logprobs_fwd(x, tokens, 9, scale)
    check_fwd(x[:9], tokens[:9], 9, scale, None, [t[:9] for t in got])
    g, ge = torch.randn(N, 2, device="cuda"), torch.randn(N, device="cuda")
    d = eas.token_logprobs_bwd(g, ge, x, tokens, got[2], got[1], scale)
    check_bwd(x[:9], tokens[:9], g[:9], ge[:9], got[2][:9], got[1][:9], scale, None, d[:9], dtype)
