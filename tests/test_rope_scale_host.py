"""Frequencies for longer contexts: what is refused before any launch (the pointers
are made up and never followed)."""
import pytest

INVALID = -1


@pytest.fixture(scope="module")
def lib():
    from verifiable_repops_gemm_gb300 import build
    return build.build()


def test_frequencies_off_their_boundary_are_refused(lib):
    from verifiable_repops_gemm_gb300 import _capi
    f = _capi.load().repops_rope_scale_frequencies_f32
    for at in (0x10000001, 0x10000002, 0x10000003):
        assert f(4, at, 2.0, 0.0, 1.0, 4.0, None) == INVALID
    for bad in ((1 << 24) + 1, 0, -1):
        assert f(bad, 0x10000000, 2.0, 0.0, 1.0, 4.0, None) == INVALID
    for bad in ((2e30, 0.0, 1.0, 4.0), (2.0, 2e30, 1.0, 4.0), (2.0, 10.0, 1.0, 2e30), (2.0, 10.0, -1.0, 4.0)):
        assert f(4, 0x10000000, *bad, None) == INVALID
