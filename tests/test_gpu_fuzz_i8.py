"""Seeded random cases of the 8-bit product, 8-bit rows and the block edge: sizes
spread over their logarithm, odd widths, pitches, offsets, storage types, missing
operands and in-place outputs, each against a statement that shares no code with
the kernels (integers, step-by-step binary32) or the library's separate operators,
bit for bit."""
import random

import numpy as np
import pytest
import torch

import rows8_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int32), b.contiguous().view(torch.int32))


def block(g, rng, rows, cols, dtype=torch.float32, scale=1.0):
    """A rows x cols block at a random place of a wider buffer."""
    pad, off = rng.choice([0, 0, 1, 3, 4, 16]), rng.choice([0, 0, 1, 4])
    buf = (torch.randn(rows, cols + pad + off, generator=g, device=DEV) * scale).to(dtype)
    return buf[:, off:off + cols]


def bytes_block(g, rng, rows, cols):
    pad, off = rng.choice([0, 0, 1, 5, 16]), rng.choice([0, 0, 1, 2, 16])
    buf = torch.randint(-128, 128, (rows * (cols + pad) + off + 1,), generator=g, device=DEV, dtype=torch.int8)
    return buf[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


@pytest.mark.parametrize("seed", range(60))
def test_products(rp, seed):
    rng = random.Random(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    M, N, K = log(rng, 1, 600), log(rng, 1, 600), log(rng, 1, 3000)
    A, B = bytes_block(g, rng, M, K), bytes_block(g, rng, N, K)
    sa = torch.rand(M, generator=g, device=DEV) + 0.1
    sb = torch.rand(N + 1, generator=g, device=DEV)[rng.randint(0, 1):][:N].contiguous()
    bias = torch.randn(N, generator=g, device=DEV) if rng.random() < 0.5 else None
    acc = (A.double() @ B.double().t()).float()                       # whole numbers: the product is exact
    want = acc * sa[:, None] * sb
    if bias is not None:
        want = want + bias
    dt = rng.choice(DTYPES)
    for cfg in (-1, 0, 1, 2):
        pad, off = rng.choice([0, 1, 3, 4, 16]), rng.choice([0, 1, 4])
        whole = torch.full((M, off + N + pad), 7.0, device=DEV, dtype=dt)
        out = whole[:, off:off + N]
        got = rp.gemm_i8(A, B.t(), sa, sb, out=out, bias=bias, config=cfg)
        assert got is out and torch.equal(out, want.to(dt)), (M, N, K, cfg, dt)
        assert bool((whole[:, :off] == 7).all()) and bool((whole[:, off + N:] == 7).all()), (M, N, K, cfg, dt)


@pytest.mark.parametrize("seed", range(40))
def test_rows(rp, seed):
    rng = random.Random(1000 + seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows, cols = log(rng, 1, 200), log(rng, 1, 3000)
    group, dt = rng.choice([0, 32, 64, 128, 256]), rng.choice(DTYPES)
    x = block(g, rng, rows, cols, dt, 10.0 ** rng.uniform(-4, 4))
    if rng.random() < 0.3:
        x[rng.randrange(rows), rng.randrange(cols)] = rng.choice([float("inf"), float("nan"), 0.0])
    q, s = rp.quantize_rows(x, group=group)
    wq, ws = ref.quantize(x.float().cpu().numpy(), group)
    assert np.array_equal(q.cpu().numpy(), wq)
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
    out = block(g, rng, rows, cols, rng.choice(DTYPES))
    rp.dequantize_rows(q, s, group=group, out=out)
    v = torch.from_numpy(ref.dequantize(wq, ws, group).copy()).to(DEV).to(out.dtype)
    assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(v)) and torch.equal(torch.isnan(out), torch.isnan(v))


@pytest.mark.parametrize("seed", range(40))
def test_backward_from_rows(rp, seed):
    rng = random.Random(2000 + seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows, cols, group = log(rng, 1, 300), log(rng, 1, 9000), rng.choice([0, 32, 64, 128, 256])
    q, s = rp.quantize_rows(block(g, rng, rows, cols, scale=2.0), group=group)
    u, us = rp.quantize_rows(block(g, rng, rows, cols, scale=2.0), group=group)
    x, xu = rp.dequantize_rows(q, s, group=group), rp.dequantize_rows(u, us, group=group)
    d, res = block(g, rng, rows, cols), block(g, rng, rows, cols) if rng.random() < 0.5 else None
    dg, du, h = (block(g, rng, rows, cols) for _ in range(3))
    rp.swiglu_backward_i8(q, s, u, us, d, dg=dg, du=du, group=group, h=h)
    wg, wu = rp.swiglu_backward(x, xu, d)
    assert same(dg, wg) and same(du, wu) and same(h, rp.swiglu(x, xu))
    gamma = torch.randn(cols, generator=g, device=DEV)
    dx, h = block(g, rng, rows, cols), block(g, rng, rows, cols)
    _, dgamma = rp.rmsnorm_backward_i8(q, s, gamma, 1e-5, d, dx=dx, group=group, res=res, h=h)
    wdx, p = rp.rmsnorm_backward(x, gamma, 1e-5, d, res=res)
    assert same(dx, wdx) and same(dgamma, rp.colsum(p)) and same(h, rp.rmsnorm_rows(x, gamma, 1e-5))


@pytest.mark.parametrize("seed", range(60))
def test_edges(rp, seed):
    rng = random.Random(3000 + seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    gates = rng.choice([0, 1, 1, 2, 5])
    rows, cols = log(rng, 1, 400), log(rng, 1, 9000)
    rows = max(1, rows // max(gates, 1)) * max(gates, 1)
    eps, alpha = rng.choice([1e-5, 1e-6]), rng.choice([1.0, 0.5, -0.3])
    x, f = block(g, rng, rows, cols), block(g, rng, rows, cols, scale=3.0)
    pre = torch.randn(cols, generator=g, device=DEV) if rng.random() < 0.8 else None
    post = torch.randn(cols, generator=g, device=DEV) if rng.random() < 0.7 else None
    gate = block(g, rng, gates, cols) if gates else None
    kw = dict(post_gain=post, gate=gate, alpha=alpha)

    spread = gate.repeat_interleave(rows // gates, 0) if gates else None
    p = rp.rmsnorm_rows(f, post, eps) if post is not None else f
    wy = (x + (p * spread if gates else p) * alpha).contiguous()
    y, h = rp.rmsnorm_residual(x, f, pre, eps, **kw)
    assert same(y, wy) and (h is None) == (pre is None)
    assert pre is None or same(h, rp.rmsnorm_rows(wy, pre, eps))

    dy = block(g, rng, rows, cols) if pre is None or rng.random() < 0.8 else None
    dh = block(g, rng, rows, cols) if pre is not None else None
    if pre is None:
        wdx, wpre = dy, None
    else:
        wdx, t = rp.rmsnorm_backward(y, pre, eps, dh, res=dy)
        wpre = rp.colsum(t)
    dt = wdx * alpha
    wdf, wpost, wgate = (dt * spread if gates else dt).contiguous(), None, None
    if gates:
        terms = (dt * p).contiguous()
        wgate = torch.stack([rp.colsum(t) for t in terms.split(rows // gates)])
    if post is not None:
        wdf, t = rp.rmsnorm_backward(f, post, eps, wdf)
        wpost = rp.colsum(t)
    in_place = dy is not None and rng.random() < 0.5
    given = dy.clone() if dy is not None else None
    got = rp.rmsnorm_residual_backward(given, dh, y if pre is not None else None, f, pre, eps, **kw,
                                       dx=given if in_place else None)
    for name, a, b in zip(("dx", "df", "dpre", "dpost", "dgate"), got, (wdx, wdf, wpre, wpost, wgate)):
        assert (a is None) == (b is None) and (a is None or same(a, b)), (name, rows, cols, gates)


def test_two_host_threads(rp):
    """Two host threads on streams of their own, every new operator at once."""
    import threading
    want, got, errors = {}, {}, []

    def work(k, out):
        g = torch.Generator(device=DEV).manual_seed(k)
        x, f = (torch.randn(200, 1000, generator=g, device=DEV) for _ in range(2))
        gain = torch.rand(1000, generator=g, device=DEV)
        w = torch.randn(300, 1000, generator=g, device=DEV)
        y, h = rp.rmsnorm_residual(x, f, gain, post_gain=gain, gate=gain)
        q, s = rp.quantize_rows(h)
        wq, ws = rp.quantize_rows(w)
        z = rp.gemm_i8(q, wq.t(), s.view(-1), ws.view(-1))
        back = rp.rmsnorm_residual_backward(h, y, y, f, gain, post_gain=gain, gate=gain)
        out[k] = [t.clone() for t in (y, h, z) + back]

    for k in (1, 2):
        work(k, want)
    torch.cuda.synchronize()

    def run(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    work(k, got)
                torch.cuda.current_stream().synchronize()
        except Exception as e:      # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in (1, 2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert all(same(a, b) for k in (1, 2) for a, b in zip(got[k], want[k]))
