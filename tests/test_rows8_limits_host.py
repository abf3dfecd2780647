"""Host-only checks of the 8-bit operators at the limits of their arguments (fake
pointers, never dereferenced)."""
import pytest

A, B, C = (0x10000000 * (i + 1) for i in range(3))


@pytest.fixture(scope="module")
def L():
    from verifiable_repops_gemm_gb300 import build, _capi
    build.build()
    return _capi.load()


def test_quantize_rows_without_columns(L):
    q = L.repops_quantize_rows_i8
    assert q(4, 0, None, 0, 0, 32, None, 0, None, 0, None) == 0          # groups of columns: no scale to write
    assert q(0, 0, None, 0, 0, 0, None, 0, None, 0, None) == 0
    assert q(4, 0, None, 0, 0, 0, None, 0, None, 1, None) == -1          # a scale a row
    assert q(4, 0, None, 0, 0, 0, None, 0, C, 0, None) == -1
    assert q(4, 0, A, 0, -1, 0, B, 0, C, 1, None) == -1
