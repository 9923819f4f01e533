"""A gradient whose rows lie between those of its logits shares no byte with them and is
taken; rows that touch them, or have another pitch, are refused (CPU only; no pointer here
is ever read)."""
import pytest
import torch

from entropy_active_span_gb300 import _lib

# calls that are taken end at the missing device
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on these pointers")

N, V, E = 4, 20, 2
X, OTHER = 1 << 24, [(i + 2) << 24 for i in range(5)]


def overlaps(lib, at, ld, ldd, n=N):
    """at: elements from the first of logits to the first of their gradient."""
    tok, glp, lse, ent, _ = OTHER
    st = lib.eas_token_logprobs_bwd(glp, None, X, ld, tok, None, lse, ent, n, V, 1, _lib.EAS_BF16, 1.0, X + E * at,
                                    ldd, None, 0, None)
    return st == _lib.EAS_ERR_INVALID_ARG and b"overlaps" in lib.eas_last_error()


def shares(at, ld, ldd, n=N):
    a = {i * ld + j for i in range(n) for j in range(V)}
    return any(at + i * ldd + j in a for i in range(n) for j in range(V))


@pytest.mark.parametrize("ld", [20, 21, 39, 40, 41, 56])
def test_rows_of_one_pitch(libeas, ld):
    for at in range(-ld * N - V, ld * N + V + 1):
        if at == 0:
            assert not overlaps(libeas, 0, ld, ld)                # in place
        elif abs(at) < (N - 1) * ld + V and abs(at) > (N - 2) * ld:
            # at the ends rows may lie beside nothing: refused by their pitch or not, never
            # taken where they share an element
            assert overlaps(libeas, at, ld, ld) or not shares(at, ld, ld)
        else:
            assert overlaps(libeas, at, ld, ld) == shares(at, ld, ld), at


def test_rows_of_two_pitches(libeas):
    assert overlaps(libeas, 20, 56, 28) and overlaps(libeas, 0, 56, 28) and overlaps(libeas, -1, 20, 21)
    assert not overlaps(libeas, 3 * 56 + V, 56, 28) and not overlaps(libeas, -3 * 28 - V, 56, 28)
