"""Rows in 8 bits on the GPU: quantising and restoring against a step-by-step
binary32 statement (bit for bit), and the backward operators that read such
rows against the library's own binary32 operators on the restored rows (bit for
bit), over odd widths, short last groups, pitches, storage types, non-finite
groups, in-place calls, side streams and captured graphs."""
import numpy as np
import pytest
import torch

from verifiable_repops_gemm_gb300 import inputs

import rows8_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SHAPES = [(1, 1), (3, 5), (2, 31), (5, 33), (9, 128), (4, 260), (7, 1023), (3, 1024), (2, 1028), (5, 2048), (2, 8192),
          (2, 8200), (1, 40000)]


def bits(a):
    return np.ascontiguousarray(a).view(np.uint32)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int32), b.contiguous().view(torch.int32))


def normal(shape, sd, seed, pad=0):
    """A float32 CUDA tensor; pad > 0: a column block of wider rows."""
    rows, cols = shape
    return inputs.normal((rows, cols + pad), sd, seed, DEV)[:, :cols]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
def test_quantize_matches_the_format(rp, rows, cols, group):
    for pad, dt in ((0, "f32"), (3, "f32"), (0, "bf16"), (4, "f16")):
        x = normal((rows, cols), 3.0, rows * 7 + cols, pad).to(DTYPES[dt])
        q, s = rp.quantize_rows(x, group=group)
        wq, ws = ref.quantize(x.float().cpu().numpy(), group)
        assert np.array_equal(q.cpu().numpy(), wq)
        assert np.array_equal(bits(s.cpu().numpy()), bits(ws))
        v = rp.dequantize_rows(q, s, group=group)
        assert np.array_equal(bits(v.cpu().numpy()), bits(ref.dequantize(wq, ws, group)))
        for name, d in DTYPES.items():
            assert torch.equal(rp.dequantize_rows(q, s, group=group, dtype=d), v.to(d)), name


@pytest.mark.parametrize("group", [0, 32, 128])
def test_quantize_error_is_within_its_bound(rp, group):
    # header: scale * (1/2 + 2^-14) of every finite value
    x = normal((64, 1000), 1.0, 5) * torch.logspace(-30, 30, 64, device=DEV)[:, None]
    q, s = rp.quantize_rows(x, group=group)
    err = (rp.dequantize_rows(q, s, group=group).double() - x.double()).abs().cpu().numpy()
    bound = np.repeat(s.cpu().numpy().astype(np.float64), group or 1000, axis=1)[:, :1000] * (0.5 + 2.0 ** -14)
    assert (err <= bound).all()
    assert int(q.abs().max()) == 127


@pytest.mark.parametrize("group", [0, 32, 256])
def test_special_values(rp, group):
    x = torch.zeros(8, 512, device=DEV)
    x[1, 3] = float("inf")
    x[2, 500] = float("nan")
    x[3, 7] = -float("inf")
    x[4, :] = 1e-40                      # below the floor of a scale
    x[5, 100] = 3.4e38
    x[6, :] = -0.0
    x[7, ::2] = 127.0                    # ties: 127 * k / 127 with halves
    x[7, 1::2] = 2.5
    q, s = rp.quantize_rows(x, group=group)
    wq, ws = ref.quantize(x.cpu().numpy(), group)
    assert np.array_equal(q.cpu().numpy(), wq)
    got = s.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ws))
    assert np.array_equal(bits(np.nan_to_num(got)), bits(np.nan_to_num(ws)))
    v = rp.dequantize_rows(q, s, group=group)
    assert torch.isnan(v[1, 3]) and torch.isnan(v[2, 500]) and torch.isnan(v[3, 7])
    assert (v[0] == 0).all() and (v[4] == 0).all() and (v[6] == 0).all()


def test_nothing_to_do_and_outputs_outside_are_left(rp):
    q, s = rp.quantize_rows(torch.empty(0, 7, device=DEV))
    assert q.shape == (0, 7) and s.shape == (0, 1)
    q, s = rp.quantize_rows(torch.empty(3, 0, device=DEV), group=32)
    assert q.shape == (3, 0) and s.shape == (3, 0)
    x = normal((5, 70), 1.0, 6)
    qbuf = torch.full((7, 80), 99, dtype=torch.int8, device=DEV)
    sbuf = torch.full((7, 6), 5.0, device=DEV)
    rp.quantize_rows(x, group=32, out=qbuf[1:6, 3:73], scale=sbuf[1:6, 2:5])
    wq, ws = ref.quantize(x.cpu().numpy(), 32)
    assert np.array_equal(qbuf[1:6, 3:73].cpu().numpy(), wq) and np.array_equal(sbuf[1:6, 2:5].cpu().numpy(), ws)
    qbuf[1:6, 3:73] = 99
    sbuf[1:6, 2:5] = 5.0
    assert (qbuf == 99).all() and (sbuf == 5.0).all()


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (5, 33), (4, 256), (7, 1023), (3, 8192), (300, 260)])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_swiglu_backward_equals_the_restored_rows(rp, rows, cols, group):
    for pad in (0, 1):
        gq, gs = rp.quantize_rows(normal((rows, cols), 2.0, 10 + cols), group=group)
        uq, us = rp.quantize_rows(normal((rows, cols), 2.0, 11 + cols), group=group)
        dh = normal((rows, cols), 1.0, 12 + cols, pad)
        g, u = rp.dequantize_rows(gq, gs, group=group), rp.dequantize_rows(uq, us, group=group)
        wdg, wdu = rp.swiglu_backward(g, u, dh)
        wh = rp.swiglu(g, u)
        h = torch.empty_like(wh)
        dg, du = rp.swiglu_backward_i8(gq, gs, uq, us, dh, group=group, h=h)
        assert same(dg, wdg) and same(du, wdu) and same(h, wh)
        d2 = dh.clone()
        dg, du = rp.swiglu_backward_i8(gq, gs, uq, us, d2, dg=d2, group=group)       # in place over dh
        assert dg is d2 and same(dg, wdg) and same(du, wdu)


def test_swiglu_backward_on_column_blocks(rp):
    """g and u as the halves of one quantised [g | u], dg and du of one matrix."""
    T, f = 33, 256
    gu = normal((T, 2 * f), 2.0, 20)
    q, s = rp.quantize_rows(gu, group=128)
    dh = normal((T, f), 1.0, 21)
    out = torch.empty(T, 2 * f, device=DEV)
    rp.swiglu_backward_i8(q[:, :f], s[:, :f // 128], q[:, f:], s[:, f // 128:], dh, dg=out[:, :f], du=out[:, f:], group=128)
    v = rp.dequantize_rows(q, s, group=128)
    wdg, wdu = rp.swiglu_backward(v[:, :f], v[:, f:], dh)
    assert same(out[:, :f], wdg) and same(out[:, f:], wdu)


def test_swiglu_backward_against_binary64_and_differences(rp):
    # per element: restoring 1 rounding, sigmoid (exp within 2 ulp, sum,
    # reciprocal) under 6 half-steps, at most 6 more products and sums, whose
    # terms' magnitude is |dh u| (sigma + |g| sigma (1 + sigma)): 32 half-steps
    gq, gs = rp.quantize_rows(normal((40, 300), 2.0, 30), group=64)
    uq, us = rp.quantize_rows(normal((40, 300), 2.0, 31), group=64)
    dh = normal((40, 300), 1.0, 32)
    dg, du = rp.swiglu_backward_i8(gq, gs, uq, us, dh, group=64)
    g, u = (rp.dequantize_rows(q, s, group=64).double().cpu().numpy() for q, s in ((gq, gs), (uq, us)))
    d = dh.double().cpu().numpy()
    sg = 1.0 / (1.0 + np.exp(-g))
    wdg, wdu = d * u * (sg + g * sg * (1 - sg)), d * g * sg
    tol = 32 * 2.0 ** -24
    assert (np.abs(dg.cpu().numpy() - wdg) <= tol * np.abs(d * u) * (sg + np.abs(g) * sg * (1 + sg))).all()
    assert (np.abs(du.cpu().numpy() - wdu) <= tol * np.abs(wdu)).all()
    e = 1e-6          # central differences of d * silu(g) * u in binary64: error e^2 and 2^-53 / e
    f = lambda a: d * a / (1 + np.exp(-a)) * u
    assert np.allclose((f(g + e) - f(g - e)) / (2 * e), wdg, rtol=0, atol=1e-8 * np.abs(d * u * (1 + np.abs(g))).max())


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (33, 33), (31, 100), (70, 1023), (64, 1024), (65, 2048), (3, 4092),
                                       (2, 8192), (3, 8193), (40, 9000), (33000, 8), (33, 32772)])
def test_rmsnorm_backward_equals_the_restored_rows(rp, rows, cols):
    for group, pad in ((128, 0), (0, 3), (32, 4)):
        q, s = rp.quantize_rows(normal((rows, cols), 1.0, 40 + cols), group=group)
        x = rp.dequantize_rows(q, s, group=group)
        gamma = inputs.normal((cols,), 1.0, 41, DEV)
        dy = normal((rows, cols), 1.0, 42 + cols, pad)
        res = normal((rows, cols), 1.0, 43 + cols, pad)
        for r in (None, res):
            wdx, p = rp.rmsnorm_backward(x, gamma, 1e-5, dy, res=r)
            h = torch.empty_like(x)
            dx, dgamma = rp.rmsnorm_backward_i8(q, s, gamma, 1e-5, dy, group=group, res=r, h=h)
            assert same(dx, wdx) and same(dgamma, rp.colsum(p)) and same(h, rp.rmsnorm_rows(x, gamma, 1e-5))
        r2 = res.clone()
        dx, _ = rp.rmsnorm_backward_i8(q, s, gamma, 1e-5, dy, dx=r2, res=r2, group=group)        # in place over res
        assert dx is r2 and same(dx, wdx)


def test_side_stream_and_captured_graph(rp):
    rows, cols = 96, 512
    q, s = rp.quantize_rows(normal((rows, cols), 1.0, 50), group=128)
    gamma = inputs.normal((cols,), 1.0, 51, DEV)
    dy = normal((rows, cols), 1.0, 52)
    wdx, wdg = rp.rmsnorm_backward_i8(q, s, gamma, 1e-5, dy, group=128)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    dx, dg = torch.empty_like(wdx), torch.empty_like(wdg)
    rp.rmsnorm_backward_i8(q, s, gamma, 1e-5, dy, dx=dx, dgamma=dg, group=128, stream=side)
    side.synchronize()
    assert same(dx, wdx) and same(dg, wdg)
    dx2, dg2 = torch.empty_like(wdx), torch.empty_like(wdg)          # a raw handle: the library's own scratch
    rp.rmsnorm_backward_i8(q, s, gamma, 1e-5, dy, dx=dx2, dgamma=dg2, group=128, stream=side.cuda_stream)
    side.synchronize()
    assert same(dx2, wdx) and same(dg2, wdg)
    graphs = []
    for k in range(2):                   # two graphs alive at once, replayed on two streams
        a, b = torch.zeros_like(wdx), torch.zeros_like(wdg)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            rp.rmsnorm_backward_i8(q, s, gamma, 1e-5, dy, dx=a, dgamma=b, group=128)
        graphs.append((gr, a, b))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for st, (gr, a, b) in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for _, a, b in graphs:
        assert same(a, wdx) and same(b, wdg)
