"""The product of 8-bit integers on the GPU: every kernel against an exact
integer product scaled step by step in binary32 (bit for bit), over odd sizes,
pitches and alignments, the extreme values -128 and 127 over whole chunks of k,
storage types, bias, non-finite scales, side streams and captured graphs."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32 = np.float32


def ints(shape, seed, lo=-128, hi=128):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g, dtype=torch.int8)


def exact_product(A, B, sa, sb, bias=None):
    """fl(fl(fl(acc) * sa) * sb) (+ bias), acc in 64-bit integers (binary64
    products of whole numbers below 2^53 are exact)."""
    acc = (A.double() @ B.double().t()).numpy()
    assert np.abs(acc).max(initial=0) < 2 ** 31
    with np.errstate(all="ignore"):
        v = acc.astype(F32) * sa.numpy()[:, None] * sb.numpy()[None, :]
        return v if bias is None else v + bias.numpy()[None, :]


def operand(X, off, pad):
    """X on the GPU in a wider buffer: first byte at offset `off`, pitch + pad."""
    r, c = X.shape
    buf = torch.full((r * (c + pad) + off + 16,), 77, dtype=torch.int8, device=DEV)
    v = buf[off:off + r * (c + pad)].view(r, c + pad)[:, :c]
    v.copy_(X)
    return v


def check(rp, M, N, K, config, off=0, pad=0, bias=False, lo=-128, hi=128):
    A, B = ints((M, K), M + K, lo, hi), ints((N, K), N + 7 * K, lo, hi)
    g = torch.Generator().manual_seed(N)
    sa, sb = torch.rand(M, generator=g) + 0.5, torch.rand(N, generator=g) * 1e-2
    bi = torch.randn(N, generator=g) if bias else None
    want = exact_product(A, B, sa, sb, bi)
    a, b = operand(A, off, pad), operand(B, (off * 3) % 16, pad)
    kw = dict(config=config, bias=bi.to(DEV) if bias else None)
    got = rp.gemm_i8(a, b.t(), sa.to(DEV), sb.to(DEV), **kw)
    assert np.array_equal(got.cpu().numpy().view(np.uint32), want.astype(F32).view(np.uint32))
    return a, b, sa.to(DEV), sb.to(DEV), got, kw


SIZES = [(1, 1, 1), (1, 16, 64), (3, 5, 7), (8, 33, 64), (9, 130, 100), (16, 64, 1000), (17, 100, 129), (33, 257, 512),
         (64, 48, 513), (65, 129, 65), (128, 256, 512), (129, 257, 577), (300, 520, 1024), (257, 64, 1537),
         (1000, 100, 2048)]


@pytest.mark.parametrize("config", [-1, 0, 1, 2])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_every_kernel_is_exact(rp, M, N, K, config):
    a, b, sa, sb, got, _ = check(rp, M, N, K, config)
    for dt in (torch.float16, torch.bfloat16):
        assert torch.equal(rp.gemm_i8(a, b.t(), sa, sb, config=config, out_dtype=dt), got.to(dt))


@pytest.mark.parametrize("config", [0, 1, 2])
@pytest.mark.parametrize("off,pad", [(0, 5), (0, 16), (1, 0), (2, 2), (4, 4), (3, 13), (15, 1)])
def test_alignment_and_pitch(rp, off, pad, config):
    check(rp, 21, 70, 203, config, off, pad, bias=True)


@pytest.mark.parametrize("config", [0, 1, 2])
@pytest.mark.parametrize("K", [512, 1024, 8192, 131071])
@pytest.mark.parametrize("va,vb", [(-128, -128), (-128, 127), (127, 127), (1, -1)])
def test_extreme_sums(rp, config, K, va, vb):
    """Every product the largest there is: partial sums reach 2^23 in a chunk
    and the result 2^14 * K < 2^31; one odd value keeps the last bit alive."""
    A, B = torch.full((3, K), va, dtype=torch.int8), torch.full((18, K), vb, dtype=torch.int8)
    A[1, K // 2] = 1
    B[5, K - 1] = 3
    A[2, ::2] = -A[2, ::2].clamp_min(-127)
    one_a, one_b = torch.ones(3), torch.ones(18)
    want = exact_product(A, B, one_a, one_b).astype(F32)
    got = rp.gemm_i8(A.to(DEV), B.to(DEV).t(), one_a.to(DEV), one_b.to(DEV), config=config)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("config", [0, 1, 2])
def test_large_random_rows(rp, config):
    """A sample of rows of a product with several tiles a CTA."""
    M, N, K = 3000, 2100, 1600
    A, B = ints((M, K), 1).to(DEV), ints((N, K), 2).to(DEV)
    sa, sb = torch.rand(M, device=DEV) + 0.5, torch.rand(N, device=DEV) + 0.5
    got = rp.gemm_i8(A, B.t(), sa, sb, config=config)
    rows = [0, 1, 127, 128, 1000, 2047, 2048, 2943, 2944, 2999]
    want = exact_product(A[rows].cpu(), B.cpu(), sa[rows].cpu(), sb.cpu()).astype(F32)
    assert np.array_equal(got[rows].cpu().numpy().view(np.uint32), want.view(np.uint32))
    ref = rp.gemm_i8(A, B.t(), sa, sb, config=0)
    assert torch.equal(got, ref)


@pytest.mark.parametrize("config", [0, 1, 2])
def test_rows_outside_are_left(rp, config):
    A, B = ints((70, 200), 3).to(DEV), ints((90, 200), 4).to(DEV)
    sa, sb = torch.ones(70, device=DEV), torch.ones(90, device=DEV)
    for dt, off in ((torch.float32, 3), (torch.bfloat16, 8), (torch.float16, 1)):
        buf = torch.full((74, 110), 9.0, dtype=dt, device=DEV)
        want = rp.gemm_i8(A, B.t(), sa, sb, config=config, out_dtype=dt)
        rp.gemm_i8(A, B.t(), sa, sb, out=buf[2:72, off:off + 90], config=config)
        assert torch.equal(buf[2:72, off:off + 90], want)
        buf[2:72, off:off + 90] = 9.0
        assert (buf == 9.0).all()


@pytest.mark.parametrize("M", [40, 100])
@pytest.mark.parametrize("K", [300, 900, 3500])
@pytest.mark.parametrize("tiles", [7, 15, 16, 23, 24, 28, 29, 36, 37, 46, 47, 76, 77, 200])
def test_every_split_of_k(rp, tiles, K, M):
    """Either side of each number of tiles at which the CTAs that share one change,
    with fewer k-steps than CTAs and more; both tile heights; C aligned and not."""
    N = 128 * tiles - 3
    g = torch.Generator(device=DEV).manual_seed(tiles)
    A, B = (torch.randint(-128, 128, (r, K), generator=g, device=DEV, dtype=torch.int8) for r in (M, N))
    sa, sb, bias = torch.rand(M, device=DEV), torch.rand(N, device=DEV), torch.randn(N, device=DEV)
    want = (A.double() @ B.double().t()).float() * sa[:, None] * sb + bias
    for ldc in (N, N + 3):
        out = torch.empty(M, ldc, device=DEV)[:, :N]
        assert torch.equal(rp.gemm_i8(A, B.t(), sa, sb, out=out, bias=bias, config=1), want)
    assert rp.device_status() == 0


@pytest.mark.parametrize("config", [0, 1, 2])
@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N", [1, 9, 11, 131, 257, 260])
def test_values_behind_a_row_are_left(rp, N, dt, config):
    """Rows that start on 16 bytes and end between them, in a wider tensor."""
    M, K = 150, 96
    A, B = ints((M, K), 5).to(DEV), ints((N, K), 6).to(DEV)
    sa, sb = torch.ones(M, device=DEV), torch.ones(N, device=DEV)
    buf = torch.full((M, (N + 31) // 16 * 16), 9.0, dtype=dt, device=DEV)
    rp.gemm_i8(A, B.t(), sa, sb, out=buf[:, :N], config=config)
    assert torch.equal(buf[:, :N], (A.double() @ B.double().t()).to(dt))
    assert (buf[:, N:] == 9.0).all()


def test_empty_and_zero_k(rp):
    e = torch.empty(0, 8, dtype=torch.int8, device=DEV)
    w = ints((5, 8), 5).to(DEV)
    assert rp.gemm_i8(e, w.t(), torch.empty(0, device=DEV), torch.ones(5, device=DEV)).shape == (0, 5)
    a, b = torch.empty(3, 0, dtype=torch.int8, device=DEV), torch.empty(5, 0, dtype=torch.int8, device=DEV)
    bias = torch.arange(5, device=DEV, dtype=torch.float32)
    for cfg in (-1, 0, 1, 2):
        y = rp.gemm_i8(a, b.t(), torch.ones(3, device=DEV), torch.ones(5, device=DEV), bias=bias, config=cfg)
        assert torch.equal(y, bias.expand(3, 5))


@pytest.mark.parametrize("config", [0, 1, 2])
def test_scales_with_nan_and_infinity(rp, config):
    A, B = ints((4, 64), 6, 1, 100).to(DEV), ints((6, 64), 7, 1, 100).to(DEV)
    sa, sb = torch.ones(4, device=DEV), torch.ones(6, device=DEV)
    sa[1], sb[3] = float("nan"), float("inf")
    y = rp.gemm_i8(A, B.t(), sa, sb, config=config)
    assert torch.isnan(y[1]).all() and torch.isinf(y[[0, 2, 3], 3]).all()
    assert torch.isfinite(y[[0, 2, 3]][:, [0, 1, 2, 4, 5]]).all()


def test_quantised_rows_multiply(rp):
    """quantize_rows and gemm_i8 together: within the two formats' error bounds
    of the binary64 product.  Each restored value is within (1/2 + 2^-14) of its
    scale, so the sum is within sum |x| eb + |w| ea + ea eb, and the scaling adds
    three roundings (the sum itself is exact)."""
    g = torch.Generator(device=DEV).manual_seed(8)
    x, w = torch.randn(37, 700, generator=g, device=DEV), torch.randn(51, 700, generator=g, device=DEV) * 0.02
    xq, xs = rp.quantize_rows(x)
    wq, wscale = rp.quantize_rows(w)
    y = rp.gemm_i8(xq, wq.t(), xs.view(-1), wscale.view(-1)).double()
    ea, eb = xs.double() * (0.5 + 2.0 ** -14), wscale.double() * (0.5 + 2.0 ** -14)
    X, W = x.double(), w.double()
    bound = X.abs().sum(1, keepdim=True) * eb.t() + ea * W.abs().sum(1) + 700 * ea * eb.t()
    assert ((y - X @ W.t()).abs() <= bound + 4 * 2.0 ** -24 * y.abs()).all()


@pytest.mark.parametrize("M", [5, 200])
def test_streams_and_captured_graphs(rp, M):
    a, b, sa, sb, want, _ = check(rp, M, 300, 640, -1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for st in (side, side.cuda_stream):              # a raw handle takes the library's own scratch
        out = torch.empty_like(want)
        torch.cuda.synchronize()
        rp.gemm_i8(a, b.t(), sa, sb, out=out, stream=st)
        side.synchronize()
        assert torch.equal(out, want)
    graphs = []
    for _ in range(2):
        out = torch.zeros_like(want)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            rp.gemm_i8(a, b.t(), sa, sb, out=out)
        graphs.append((gr, out))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for st, (gr, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, out in graphs)


def test_binding_refusals(rp):
    A, W = ints((4, 32), 9).to(DEV), ints((6, 32), 10).to(DEV)
    sa, sb = torch.ones(4, device=DEV), torch.ones(6, device=DEV)
    with pytest.raises(ValueError):
        rp.gemm_i8(A, W.t().contiguous(), sa, sb)            # k not contiguous
    with pytest.raises(ValueError):
        rp.gemm_i8(A, W[:, :31].t(), sa, sb)
    with pytest.raises(TypeError):
        rp.gemm_i8(A.float(), W.t(), sa, sb)
    with pytest.raises(ValueError):
        rp.gemm_i8(A, W.t(), sb, sb)
    with pytest.raises(ValueError):
        rp.gemm_i8(A, W.t(), sa, sb.double())
    with pytest.raises(ValueError):
        rp.gemm_i8(A.cpu(), W.t(), sa, sb)
    with pytest.raises(rp.RepopsError):
        rp.gemm_i8(A, W.t(), sa, sb, config=9)
