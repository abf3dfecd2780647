"""Host-only checks of the 8-bit row and block-edge operators: refusals before
anything is launched (fake pointers, never dereferenced), and the binary64
statement the GPU tests use, its gradients against differences."""
import ctypes

import numpy as np
import pytest

import rows8_ref as ref

A, B, C, D, E, F, G, H, W = (0x10000000 * (i + 1) for i in range(9))
f32 = ctypes.c_float


@pytest.fixture(scope="module")
def L():
    from verifiable_repops_gemm_gb300 import build, _capi
    build.build()
    return _capi.load()


def test_quantize_refusals(L):
    q = L.repops_quantize_rows_i8
    ok = [4, 64, A, 0, 64, 32, B, 64, C, 2, None]

    def with_(**kw):
        v = list(ok)
        for k, x in kw.items():
            v[int(k[1:])] = x
        return q(*v)

    assert with_(_0=-1) == -1 and with_(_1=-1) == -1 and with_(_1=1 << 31) == -1
    assert with_(_2=None) == -1 and with_(_6=None) == -1 and with_(_8=None) == -1
    assert with_(_3=7) == -1
    assert with_(_4=63) == -1 and with_(_7=63) == -1 and with_(_9=1) == -1          # short pitches
    for g in (-1, 1, 16, 48, 512):
        assert with_(_5=g) == -1
    assert with_(_6=A + 16) == -2 and with_(_8=A) == -2 and with_(_8=B + 64) == -2
    assert with_(_0=1 << 60) == -1                                                  # overflowing span
    assert with_(_0=0) == 0 and with_(_1=0) == 0
    d = L.repops_dequantize_rows_i8
    assert d(4, 64, A, 64, B, 2, 32, C, 5, 64, None) == -1
    assert d(4, 64, A, 64, B, 1, 32, C, 0, 64, None) == -1
    assert d(4, 64, A, 64, B, 2, 33, C, 0, 64, None) == -1
    assert d(4, 64, A, 64, B, 2, 32, A + 8, 0, 64, None) == -2
    assert d(4, 64, A, 64, B, 2, 32, None, 0, 64, None) == -1


def test_swiglu_backward_refusals(L):
    s = L.repops_swiglu_backward_i8

    def call(**kw):
        a = dict(rows=4, cols=64, g=A, ldg=64, gs=B, ldgs=2, u=C, ldu=64, us=D, ldus=2, group=32, dh=E, lddh=64, dg=F,
                 lddg=64, du=G, lddu=64, h=H, ldh=64)
        a.update(kw)
        return s(*a.values(), None)

    assert call(rows=-1) == -1 and call(group=31) == -1 and call(cols=1 << 31) == -1
    for k in ("g", "gs", "u", "us", "dh", "dg", "du"):
        assert call(**{k: None}) == -1
    for k in ("ldg", "ldu", "lddh", "lddg", "lddu", "ldh"):
        assert call(**{k: 63}) == -1
    assert call(ldgs=1) == -1 and call(ldus=1) == -1
    for k in ("dg", "du", "h"):
        for other in (A, B, C, D):
            assert call(**{k: other}) == -2
        assert call(**{k: E + 16}) == -2                     # dh, but not in place
    assert call(dg=F, du=F) == -2 and call(h=G + 64) == -2
    assert call(dg=E, du=E) == -2                            # only one output may be dh
    assert call(rows=0) == 0


def test_rmsnorm_backward_refusals(L):
    s = L.repops_rmsnorm_backward_i8
    need = L.repops_rmsnorm_backward_i8_workspace_bytes(4, 64)
    assert need > 0 and L.repops_rmsnorm_backward_i8_workspace_bytes(0, 64) == 0

    def call(**kw):
        a = dict(rows=4, cols=64, x=A, ldx=64, xs=B, lds=2, group=32, gamma=C, eps=f32(1e-5), dy=D, lddy=64, res=E,
                 ldres=64, dx=F, lddx=64, h=G, ldh=64, dgamma=H, ws=W, wsb=need)
        a.update(kw)
        return s(*a.values(), None)

    assert call(rows=-1) == -1 and call(group=5) == -1
    for k in ("x", "xs", "gamma", "dy", "dx", "dgamma"):
        assert call(**{k: None}) == -1
    for k in ("ldx", "lddy", "ldres", "lddx", "ldh"):
        assert call(**{k: 63}) == -1
    assert call(lds=1) == -1
    assert call(wsb=need - 1) == -1 and call(ws=W + 4) == -1
    for k in ("dx", "h", "dgamma"):
        for other in (A, B, C, D, W):
            assert call(**{k: other}) == -2, (k, other)
    assert call(dx=E, lddx=68) == -2 and call(h=E) == -2 and call(h=F) == -2 and call(dgamma=F + 8) == -2
    for other in (A, B, C, D, E):
        assert call(ws=other) == -2                          # scratch over an input
    assert call(cols=400000, ldx=400000, lds=12500, lddy=400000, ldres=400000, lddx=400000, ldh=400000) == -7
    assert call(rows=0) == 0


def test_edge_refusals(L):
    s = L.repops_rmsnorm_residual_f32

    def call(**kw):
        a = dict(rows=4, cols=64, x=A, ldx=64, f=B, ldf=64, post=C, gate=D, ldgate=64, per=2, alpha=f32(1), pre=E,
                 eps=f32(1e-5), y=F, ldy=64, h=G, ldh=64)
        a.update(kw)
        return s(*a.values(), None)

    assert call(rows=-1) == -1 and call(cols=-1) == -1
    for k in ("x", "f", "y", "h", "pre"):
        assert call(**{k: None}) == -1
    for k in ("ldx", "ldf", "ldgate", "ldy", "ldh"):
        assert call(**{k: 63}) == -1
    assert call(per=0) == -1 and call(per=3) == -1
    for k in ("y", "h"):
        for other in (C, D, E):
            assert call(**{k: other}) == -2
        assert call(**{k: A + 4}) == -2 and call(**{k: B + 4}) == -2
    assert call(y=A, ldy=68) == -2                           # in place only with the same pitch
    assert call(y=A, h=A) == -2 and call(y=F, h=F + 64) == -2
    big = 400000
    assert call(cols=big, ldx=big, ldf=big, ldgate=big, ldy=big, ldh=big) == -7
    assert call(rows=0) == 0 and call(cols=0) == 0


def test_edge_backward_refusals(L):
    s = L.repops_rmsnorm_residual_backward_f32
    ws_bytes = L.repops_rmsnorm_residual_backward_workspace_bytes
    need = ws_bytes(4, 64, 2)
    assert need > 0 and ws_bytes(4, 64, 3) == 0 and ws_bytes(4, 64, -1) == 0
    ptr = {k: 0x10000000 * (i + 1) for i, k in enumerate(
        ("dy", "dh", "y", "f", "post", "gate", "pre", "dx", "df", "dpre", "dpost", "dgate", "ws"))}

    def call(**kw):
        p = ptr
        a = dict(rows=4, cols=64, dy=p["dy"], lddy=64, dh=p["dh"], lddh=64, y=p["y"], ldy=64, f=p["f"], ldf=64,
                 post=p["post"], gate=p["gate"], ldgate=64, per=2, alpha=f32(1), pre=p["pre"], eps=f32(1e-5),
                 dx=p["dx"], lddx=64, df=p["df"], lddf=64, dpre=p["dpre"], dpost=p["dpost"], dgate=p["dgate"],
                 lddgate=64, ws=p["ws"], wsb=need)
        a.update(kw)
        return s(*a.values(), None)

    assert call(rows=-1) == -1
    for k in ("dh", "y", "f", "post", "gate", "pre", "dx", "df", "dpre", "dpost", "dgate"):
        assert call(**{k: None}) == -1, k
    assert call(dy=None, dh=None, y=None, pre=None, dpre=None) == -1
    for k in ("lddy", "lddh", "ldy", "ldf", "ldgate", "lddx", "lddf", "lddgate"):
        assert call(**{k: 63}) == -1, k
    assert call(per=0) == -1 and call(per=3) == -1
    assert call(wsb=need - 1) == -1 and call(ws=ptr["ws"] + 8) == -1
    outs = ("dx", "df", "dpre", "dpost", "dgate")
    for o in outs:
        for i in ("dy", "dh", "y", "f", "post", "gate", "pre", "ws"):
            if (o, i) != ("dx", "dy"):
                assert call(**{o: ptr[i]}) == -2, (o, i)
        for p in outs:
            if p != o:
                assert call(**{o: ptr[p]}) == -2, (o, p)
    assert call(dx=ptr["dy"], lddx=68) == -2
    for i in ("dy", "dh", "y", "f", "post", "gate", "pre"):
        assert call(ws=ptr[i]) == -2, i                      # scratch over an input
    assert call(rows=0) == 0


def test_binary64_gradients_against_differences():
    """The reference's gradients against central differences of its forward:
    step 1e-5, error about step^2 and 2^-53 / step relative to the loss terms."""
    rng = np.random.default_rng(3)
    rows, cols, gates, alpha, eps = 4, 7, 2, 0.6, 1e-5
    x, f, dy, dh = (rng.normal(size=(rows, cols)) for _ in range(4))
    post, pre = 1 + 0.1 * rng.normal(size=cols), 1 + 0.1 * rng.normal(size=cols)
    gate = 0.5 + 0.2 * rng.normal(size=(gates, cols))

    def loss(x, f, post, gate, pre):
        y, h = ref.edge64(x, f, post, np.repeat(gate, rows // gates, axis=0), alpha, pre, eps)
        return (dy * y).sum() + (dh * h).sum()

    args = {"dx": x, "df": f, "dpost": post, "dgate": gate, "dpre": pre}
    y, _ = ref.edge64(x, f, post, np.repeat(gate, rows // gates, axis=0), alpha, pre, eps)
    got = ref.edge_backward64(dy, dh, y, f, post, np.repeat(gate, rows // gates, axis=0), alpha, pre, eps, gates)
    for name, a in args.items():
        num = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            keep = a[i]
            v = []
            for e in (1e-5, -1e-5):
                a[i] = keep + e
                v.append(loss(x, f, post, gate, pre))
            a[i] = keep
            num[i] = (v[0] - v[1]) / 2e-5
        assert np.allclose(num, got[name][0], rtol=0, atol=1e-7), name


def test_reference_format_on_known_values():
    q, s = ref.quantize(np.array([[127.0, -63.5, 1.0, 0.5]], np.float32), 0)
    assert s[0, 0] == 1.0 and q.tolist() == [[127, -64, 1, 0]]
    q, s = ref.quantize(np.array([[0.0, 0.0]], np.float32), 32)
    assert q.tolist() == [[0, 0]] and s[0, 0] > 0


def test_gemm_i8_refusals(L):
    s = L.repops_gemm_i8
    assert L.repops_gemm_i8_config_count() == 3
    ws_bytes = L.repops_gemm_i8_workspace_bytes
    need = ws_bytes(1, 4, 6, 64)
    assert need > 0 and ws_bytes(0, 4, 6, 64) == 0 and ws_bytes(9, 4, 6, 64) == 0 and ws_bytes(1, 0, 6, 64) == 0
    assert L.repops_gemm_i8_auto_config(-1, 1, 1) == -1

    def call(**kw):
        a = dict(cfg=1, M=4, N=6, K=64, A=A, lda=64, sa=B, B=C, ldb=64, sb=D, bias=E, C=F, tc=0, ldc=6, ws=W, wsb=need)
        a.update(kw)
        return s(*a.values(), None)

    assert call(M=-1) == -1 and call(N=-1) == -1 and call(K=-1) == -1
    assert call(cfg=3) == -1 and call(cfg=-2) == -1 and call(tc=3) == -1
    for k in ("A", "sa", "B", "sb", "C"):
        assert call(**{k: None}) == -1
    assert call(lda=63) == -1 and call(ldb=63) == -1 and call(ldc=5) == -1
    assert call(wsb=need - 1) == -1 and call(ws=W + 8) == -1
    for other in (A, B, C, D, E):
        assert call(C=other) == -2
        assert call(ws=other) == -2
    assert call(ws=F) == -2
    assert call(K=131072, lda=131072, ldb=131072) == -7
    assert call(M=0) == 0 and call(N=0) == 0


def test_binding_refuses_rows_that_share_memory():
    """An expanded tensor's rows are one row in memory: reading or writing them at
    a pitch of their width would leave it."""
    import torch

    import verifiable_repops_gemm_gb300 as rp
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2)
    assert rp._rows_i8(q, s, 32, "q")[1::2] == (64, 2)
    assert rp._rows_i8(q[:1].expand(1, 64), s[:1], 32, "q")[1] == 64
    assert rp._rows_i8(q[:, :60], s, 32, "q")[1] == 64
    with pytest.raises(ValueError):
        rp._rows_i8(q[:1].expand(4, 64), s, 32, "q")
    with pytest.raises(ValueError):
        rp._rows_i8(q, s[:1].expand(4, 2), 32, "q")
    with pytest.raises(ValueError):
        rp._pitch(torch.zeros(1).expand(4, 1), "x")
    with pytest.raises(ValueError):
        rp._rows_i8(q, s, 48, "q")
    with pytest.raises(ValueError):
        rp._rows_i8(q.t(), s, 32, "q")
    assert rp._pitch(torch.zeros(0, 5).expand(0, 5), "x") == 5
