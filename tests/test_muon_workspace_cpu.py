"""Sizes of the orthogonalised update's workspace, as the header gives them (CPU only)."""
import pytest


def up(x):
    return (x + 63) // 64 * 64


@pytest.mark.parametrize("L,n,m", [(65535, 1, 1), (65535, 7, 3), (1000, 128, 384), (12, 384, 128), (1, 1, 512)])
def test_small_matrices_keep_to_the_status_word(libeas, L, n, m):
    assert 16 <= libeas.eas_orthogonalize_workspace_size(L, n, m) <= (1024 if m <= 384 else 1024 + (L << 16))


@pytest.mark.parametrize("L,n,m,each", [(1, 128, 385, 32768), (300, 448, 100, 32768), (7, 2, 449, 65536), (20, 128, 512, 65536)])
def test_small_matrices_that_leave_shared_memory(libeas, L, n, m, each):
    size = libeas.eas_orthogonalize_workspace_size(L, n, m)
    assert L * each <= size <= 1024 + L * each


@pytest.mark.parametrize("L,n,m", [(1, 129, 129), (1, 128, 513), (3, 1, 6000), (1, 129, 8000), (200, 130, 130), (8, 1024, 2048),
                                   (1, 4096, 4096), (1, 640, 8192), (30, 128, 900), (1, 65536, 129), (2, 65536, 65536)])
def test_larger_ones(libeas, L, n, m):
    size = libeas.eas_orthogonalize_workspace_size
    n, m = min(n, m), max(n, m)
    own = L * (8 * n * up(m) + 4 * n * up(n))
    assert size(L, n, m) == size(L, m, n)
    assert own <= size(L, n, m) <= 1.02 * own + (5 << 20)
