"""The RMS norm takes every positive eps (CPU only; no pointer here is ever read): the
next check, a missing weight, is what refuses."""
import pytest

from entropy_active_span_gb300 import _lib

A, B, C, D = ((i + 1) << 24 for i in range(4))


@pytest.mark.parametrize("eps", [1e-44, 2e-38, 1e-35, 9e-31, 1e-30, 1e30])
def test_small_eps_is_not_refused(libeas, eps):
    calls = (lambda e: libeas.eas_rmsnorm_fwd(A, None, None, None, 4, 64, _lib.EAS_BF16, e, None, B, None, None, None),
             lambda e: libeas.eas_rmsnorm_bwd(A, B, None, None, None, 4, 64, _lib.EAS_BF16, e, C, D, None, 0, None))
    for call in calls:
        assert call(eps) == _lib.EAS_ERR_INVALID_ARG and b"null pointer" in libeas.eas_last_error()
        assert call(0.0) == _lib.EAS_ERR_INVALID_ARG and b"eps" in libeas.eas_last_error()
