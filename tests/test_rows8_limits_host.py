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


def test_gemm_i8_scratch_sizes(L):
    """Aligned weights are read where they lie: the scratch of the tensor-core
    kernels is the widened tokens (and, with thousands of them, the widened weights);
    others are copied."""
    ws, op = L.repops_gemm_i8_workspace_bytes, L.repops_gemm_i8_operand_workspace_bytes
    assert ws(1, 64, 8192, 8192) == 64 * 8192 * 2 == op(1, 64, 8192, 8192, A, 8192) == op(1, 64, 8192, 8192, None, 0)
    for b, ldb in ((A + 1, 8192), (A, 8193), (A + 8, 8200)):
        assert op(1, 64, 8192, 8192, b, ldb) == 64 * 8192 * 2 + 8192 * 8192
        assert op(2, 64, 8192, 8192, b, ldb) == ws(2, 64, 8192, 8192) == (64 + 8192) * 8192 * 2
        assert op(0, 64, 8192, 8192, b, ldb) == 0
        auto = L.repops_gemm_i8_auto_config(64, 8192, 8192)
        assert op(-1, 64, 8192, 8192, b, ldb) == op(auto, 64, 8192, 8192, b, ldb)
    for bad in ((3, 4, 6, 64), (1, 0, 6, 64), (1, 4, 6, 0), (1, 4, 6, 131072), (1, -4, 6, 64)):
        assert ws(*bad) == 0 == op(*bad, A + 1, 64)


def test_gemm_i8_scratch_refusals(L):
    s = L.repops_gemm_i8
    D, E, F, W = (0x10000000 * (i + 4) for i in range(4))
    need = L.repops_gemm_i8_workspace_bytes(1, 4, 6, 64)
    full = L.repops_gemm_i8_operand_workspace_bytes(1, 4, 6, 64, C + 1, 64)
    assert full == need + 6 * 128

    def call(**kw):
        a = dict(cfg=1, M=4, N=6, K=64, A=A, lda=64, sa=B, B=C + 1, ldb=64, sb=D, bias=E, C=F, tc=0, ldc=6, ws=W, wsb=full)
        a.update(kw)
        return s(*a.values(), None)

    assert call(wsb=need - 1) == -1 and call(ws=W + 8) == -1
    for other in (A, B, C, D, E, F):
        assert call(ws=other - need) == -2                   # the copy's part over an operand
        assert call(ws=other, wsb=need) == -2
