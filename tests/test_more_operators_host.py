"""Host-only checks of the AdamW, head-norm and log-probability entry points: what
they refuse before any CUDA call (the pointers are made up and never followed), the
words of an AdamW step, and the tests' own statements of the 8-bit codes."""
import ctypes

import numpy as np
import pytest

import adamw_ref
import logprobs_ref

OK, INVALID, ALIAS, ORDER, UNSUPPORTED = 0, -1, -2, -3, -7
A, B, C, D, E, F, G, H = (0x10000000 * i for i in range(1, 9))


@pytest.fixture(scope="module")
def L():
    from verifiable_repops_gemm_gb300 import build, _capi
    build.build()
    return _capi.load()


def ptrs(*p):
    return (ctypes.c_uint64 * max(len(p), 1))(*p)


def doubles(*v):
    return (ctypes.c_double * len(v))(*v)


def test_adamw_scalars(L):
    w = np.zeros(4, np.uint32)
    for step, lr, b1, b2, seed in ((1, 1e-3, 0.9, 0.999, 0), (7, 3e-4, 0.9, 0.95, 5), (100000, 0.0, 0.0, 0.0, 1 << 31),
                                   (1 << 40, 1.0, 0.99999, 0.999999, 3)):
        assert L.repops_adamw_scalars(step, doubles(lr, b1, b2), seed, w.ctypes.data) == OK
        want = adamw_ref.scalars(step, lr, (b1, b2), seed)
        # beta^step by squaring is off by a few roundings of binary64
        assert np.allclose(w[:3].view(np.float32), np.array(want[:3], np.float64), rtol=2.0 ** -23, atol=0)
        assert int(w[3]) == want[3]
    for bad in ((0, 1e-3, 0.9, 0.9), (1, 1e-3, 1.0, 0.9), (1, 1e-3, 0.9, -0.1), (1, float("nan"), 0.9, 0.9),
                (1, float("inf"), 0.9, 0.9), (1, 1e-3, float("nan"), 0.9)):
        assert L.repops_adamw_scalars(bad[0], doubles(*bad[1:]), 0, w.ctypes.data) == INVALID
    assert L.repops_adamw_scalars(1, doubles(1e-3, 0.9, 0.9), 0, None) == INVALID
    assert L.repops_adamw_scalars(1, None, 0, w.ctypes.data) == INVALID


def test_adamw_refuses(L):
    n2 = (ctypes.c_int64 * 2)(100, 50)
    words = (ctypes.c_uint32 * 4)()
    one = (ctypes.c_int * 2)(0, 1)

    def call(tensors=2, sizes=n2, theta=ptrs(A, B), k=1, grads=ptrs(C, D), kind=0, order=one, m=ptrs(E, E + 400),
             v=ptrs(F, F + 400), ms=None, vs=None, b1=0.9, b2=0.99, eps=1e-8, scalars=words):
        return L.repops_adamw(tensors, sizes, theta, k, grads, kind, order, m, v, ms, vs, None, doubles(b1, b2, eps), scalars, 0,
                              None, None)

    assert call(tensors=0) == OK
    assert call(sizes=(ctypes.c_int64 * 2)(0, 0)) == OK                # nothing in either
    assert call(tensors=-1) == INVALID
    assert call(k=0) == INVALID
    assert call(k=1025) == INVALID
    assert call(kind=3) == INVALID
    assert call(sizes=(ctypes.c_int64 * 2)(100, -1)) == INVALID
    assert call(sizes=(ctypes.c_int64 * 2)(100, 1 << 41)) == INVALID
    assert call(theta=ptrs(A, 0)) == INVALID
    assert call(grads=ptrs(0, D)) == INVALID
    assert call(m=ptrs(E, 0)) == INVALID
    assert call(ms=ptrs(G, G + 1)) == INVALID                          # one scale without the other
    assert call(scalars=None) == INVALID
    assert call(theta=ptrs(A + 2, B)) == INVALID                       # off its elements' boundary
    assert call(m=ptrs(E, E + 402)) == INVALID and call(v=ptrs(F + 1, F + 400)) == INVALID
    assert call(grads=ptrs(C, D + 1), kind=1) == INVALID and call(grads=ptrs(C + 2, D)) == INVALID
    assert call(eps=-1.0) == INVALID
    assert call(eps=float("nan")) == INVALID
    assert call(b1=1.0) == INVALID
    assert call(k=2, grads=ptrs(C, C, D, D), order=(ctypes.c_int * 2)(0, 0)) == ORDER
    assert call(k=2, grads=ptrs(C, C, D, D), order=(ctypes.c_int * 2)(0, 2)) == ORDER
    assert call(theta=ptrs(A, A)) == ALIAS                             # the same tensor twice
    assert call(theta=ptrs(A, A + 396)) == ALIAS                       # by its last element
    assert call(grads=ptrs(A, D)) == ALIAS
    assert call(grads=ptrs(B + 196, D)) == ALIAS                       # another tensor's last element
    assert call(m=ptrs(E, E + 396)) == ALIAS
    assert call(v=ptrs(E, F)) == ALIAS
    assert call(m=ptrs(E, E + 100), v=ptrs(F, F + 100), ms=ptrs(G, G), vs=ptrs(H, H + 1)) == ALIAS
    # scalars on the device inside a tensor that is written
    assert L.repops_adamw(2, n2, ptrs(A, B), 1, ptrs(C, D), 0, one, ptrs(E, E + 400), ptrs(F, F + 400), None, None, None,
                          doubles(0.9, 0.99, 1e-8), A, 1, None, None) == ALIAS
    assert L.repops_adamw(2, n2, ptrs(A, B), 1, ptrs(C, D), 0, one, ptrs(E, E + 400), ptrs(F, F + 400), None, None, None,
                          doubles(0.9, 0.99, 1e-8), words, 0, B, None) == ALIAS
    mo = L.repops_adamw_moments
    assert mo(0, None, None, None, None, None, None, None) == OK
    assert mo(-1, A, B, C, D, E, F, None) == INVALID
    assert mo(10, A, B, C, None, E, F, None) == INVALID
    assert mo(10, A, B, C, D, E + 2, F, None) == INVALID
    assert mo(10, A, B, C, D, E, E + 36, None) == ALIAS
    assert mo(10, A, B, C, D, A + 8, F, None) == ALIAS


def test_logprobs_refuse(L):
    def call(rows=4, cols=100, x=A, kind=0, ld=100, t=B, T=1.0, top=0, logp=C, lse=C + 16, ent=C + 32, stats=D, tl=None,
             ti=None):
        return L.repops_token_logprobs(rows, cols, x, kind, ld, t, T, top, logp, lse, ent, stats, tl, ti, None)

    assert call(rows=0) == OK
    for bad in (dict(rows=-1), dict(cols=0), dict(kind=9), dict(ld=99), dict(x=None), dict(x=A + 2), dict(logp=None),
                dict(stats=None), dict(stats=D + 4), dict(T=0.0), dict(T=-1.0), dict(T=float("nan")), dict(T=1e7),
                dict(top=-1), dict(top=101), dict(top=3), dict(top=3, tl=E), dict(ld=1 << 62), dict(t=B + 4),
                dict(logp=C + 2), dict(lse=C + 17), dict(ent=C + 34), dict(top=2, tl=E + 1, ti=F),
                dict(top=2, tl=E, ti=F + 4)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(top=33, tl=E, ti=F), dict(cols=16384001, ld=16384001), dict(rows=(1 << 27) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(logp=A + 1596), dict(lse=C), dict(stats=B), dict(top=2, tl=C, ti=F), dict(top=2, tl=E, ti=A)):
        assert call(**bad) == ALIAS, bad

    def back(rows=4, cols=100, x=A, kind=0, ld=100, t=B, T=1.0, st=D, dl=E, de=None, dx=F, ldd=100):
        return L.repops_token_logprobs_backward(rows, cols, x, kind, ld, t, T, st, dl, de, dx, ldd, None)

    assert back(rows=0) == OK
    for bad in (dict(rows=-1), dict(cols=0), dict(kind=-1), dict(dl=None), dict(t=None), dict(st=None), dict(st=D + 8),
                dict(dx=None), dict(dx=F + 1), dict(ldd=99), dict(T=0.0), dict(t=B + 2), dict(dl=E + 1), dict(de=G + 2)):
        assert back(**bad) == INVALID, bad
    for bad in (dict(dx=A, ldd=101), dict(dx=A + 400), dict(dx=D), dict(dx=E), dict(dx=B), dict(de=F + 16)):
        assert back(**bad) == ALIAS, bad


def test_head_norm_rope_refuses(L):
    def call(rows=4, q=2, k=1, dim=64, x=A, kind=0, ldx=192, qg=B, kg=B + 256, cos=C, sin=D, pairs=32, positions=50,
             layout=0, inverse=0, pos=None, wide=0, first=0, period=4, y=E, ldy=192):
        return L.repops_head_norm_rope(rows, q, k, dim, x, kind, ldx, qg, kg, 1e-6, cos, sin, pairs, positions, layout,
                                       inverse, pos, wide, first, period, y, ldy, None)

    assert call(rows=0) == OK and call(q=0, k=0, qg=None, kg=None, ldx=0, ldy=0) == OK
    for bad in (dict(rows=-1), dict(q=-1), dict(dim=0), dict(kind=4), dict(ldx=191), dict(ldy=191), dict(x=None),
                dict(y=None), dict(x=A + 2), dict(qg=None), dict(kg=None), dict(inverse=1), dict(pairs=33), dict(pairs=-1),
                dict(cos=None), dict(positions=0), dict(layout=2), dict(first=-1), dict(period=0), dict(first=47),
                dict(pos=F, wide=2), dict(pos=F + 2), dict(pos=F + 4, wide=1), dict(qg=B + 2), dict(kg=B + 258),
                dict(cos=C + 1), dict(sin=D + 2)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dim=513, ldx=1539, ldy=1539), dict(positions=1 << 31), dict(q=65537, ldx=1 << 24, ldy=1 << 24)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(y=A, ldy=193), dict(y=A + 4), dict(y=B), dict(y=C), dict(y=D), dict(pos=E)):
        assert call(**bad) == ALIAS, bad

    def back(rows=4, q=2, k=1, dim=64, dy=F, x=A, ld=192, qg=B, kg=B + 256, pairs=32, dx=E, dq=G, dk=G + 256, ws=H,
             wsb=1 << 20, lddx=192):
        return L.repops_head_norm_rope_backward(rows, q, k, dim, dy, 0, ld, x, ld, qg, kg, 1e-6, C, D, pairs, 50, 0, None, 0, 0,
                                                4, dx, lddx, dq, dk, ws, wsb, None)

    assert back(rows=0) == OK
    for bad in (dict(qg=None), dict(dk=None), dict(q=0, ld=64), dict(dy=None), dict(x=None), dict(dx=None), dict(ws=H + 4),
                dict(wsb=100), dict(pairs=40)):
        assert back(**bad) == INVALID, bad
    for bad in (dict(dx=A), dict(dx=F, lddx=200), dict(dq=G, dk=G + 252), dict(dq=B), dict(ws=A), dict(dx=C), dict(dq=H)):
        assert back(**bad) == ALIAS, bad
    need = L.repops_head_norm_rope_backward_workspace_bytes
    assert need(-1, 2, 1, 64) == 0 and need(4, 2, 1, 64) == 2 * 64 * 4
    # every level of the sums above the 32768 results the last fold takes fits: a 32nd of
    # the one below, rounded up
    for rows in (1, 31, 5000, 40000, 140000, 1 << 20, 1 << 26):
        q, total = -(-rows * 8 // 32), 0
        n = q
        while n > 32768:
            n = -(-n // 32)
            total += n
        assert need(rows, 8, 0, 64) >= (q + total) * 64 * 4
    f = L.repops_rope_scale_frequencies_f32
    for bad in ((0, A, 2.0, 0.0, 1.0, 4.0), (4, None, 2.0, 0.0, 1.0, 4.0), (4, A, 0.0, 0.0, 1.0, 4.0),
                (4, A, 2.0, 10.0, 4.0, 4.0), (4, A, 2.0, -1.0, 1.0, 4.0), (4, A, float("nan"), 0.0, 1.0, 4.0)):
        assert f(*bad, None) == INVALID


def test_the_references_agree_with_their_formats():
    """The 8-bit codes of the tests against a list of every code's value, and e(x) and
    ln against NumPy's."""
    rng = np.random.default_rng(1)
    codes = np.arange(256)
    e, f = codes >> 4, codes & 15
    root = np.where(e == 0, f / 16 * 2.0 ** -14, (1 + f / 16) * 2.0 ** (e - 15.0))
    e, f = (codes[:127] >> 3), codes[:127] & 7
    mant = np.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7.0))
    x = np.exp(rng.standard_normal(1280) * 4).astype(np.float32)
    for is_root, grid in ((False, mant), (True, root)):
        for d in (0.0, 65535.0):
            v, s = adamw_ref.coded(x, is_root, np.full(1280, d))
            unit = np.repeat(2.0 ** (s.astype(np.float64) - 127), 128)
            at = x / unit
            below = np.searchsorted(grid, at, side="right") - 1
            want = grid[below] if d == 0 else grid[np.minimum(below + (at > grid[below]), len(grid) - 1)]
            if is_root:
                want = np.maximum(want, grid[1])
            # with all of the dither set only a cut-off part below 2^-17 of a code stays down
            assert np.mean(v == (want * unit).astype(np.float32)) > 0.999
            assert (np.abs(at - v / unit) <= np.diff(grid, append=2 * grid[-1])[below]).all()
    z = -np.abs(rng.standard_normal(20000) * 30).astype(np.float32)
    got, t = logprobs_ref.exp_t(z, np.float32(0), np.float32(logprobs_ref.LOG2E))
    want = np.exp(z.astype(np.float64))
    keep = z > -87
    assert (np.abs(got[keep] / want[keep] - 1) <= logprobs_ref.E_REL + np.abs(z[keep]) * 3 * 2.0 ** -24).all()
    assert (got[z < -88.1] == 0).all()
    for s in (0.5, 1.0, 1.4142135623730951, 1.5, 2.0, 131072.7, 3e38):
        want = np.log(np.float64(np.float32(s)))
        assert abs(logprobs_ref.ln_fixed(s) - want) <= 2.0 ** -22 * abs(want)


def test_models_refuse_what_they_lack():
    import torch
    from verifiable_repops_gemm_gb300 import decoder, train
    cfg = decoder.DecoderConfig(d=32, heads=2, kv_heads=2, ffn=32, seq_len=8)
    model = train.Model(cfg, 1, "cpu")
    with pytest.raises(ValueError):
        train.token_gradient(model, torch.zeros(8, 32), torch.zeros(8, dtype=torch.int64), model.gradient_buffer(), None)
    with pytest.raises(ValueError):
        train.AdamW(model, 1e-3, bits=16)
    for bad in (-2, 3, 18):
        with pytest.raises(ValueError):
            decoder.rope_tables(decoder.DecoderConfig(d=32, heads=2, kv_heads=2, ffn=32, seq_len=8, rope_base=10000.0,
                                                      rope_dim=bad), "cpu")
