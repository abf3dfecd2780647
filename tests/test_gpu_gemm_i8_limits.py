"""The 8-bit product at the limits of its arguments: scratch of exactly the size
asked for, whatever the weights' alignment, and more tokens than a grid's y
dimension has tiles."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def ints(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8).to(DEV)


@pytest.mark.parametrize("config", [0, 1, 2])
@pytest.mark.parametrize("offset", [0, 3])
def test_scratch_of_the_size_asked_for(rp, config, offset):
    """Config 1 reads aligned weights where they lie: its scratch is the widened
    tokens alone.  Other weights' copy comes from longer scratch, or from the
    library's pool."""
    M, N, K = 40, 300, 640
    L = rp.load()
    a = ints((M, K), 1)
    b = ints((N, K + 16), 2)[:, offset:offset + K]
    sa, sb = torch.rand(M, device=DEV) + 0.5, torch.rand(N, device=DEV) + 0.5
    want = rp.gemm_i8(a, b.t(), sa, sb, config=0)
    assert torch.equal(want, (a.double() @ b.double().t()).float() * sa[:, None] * sb)      # |sums| < 2^24: exact
    short = L.repops_gemm_i8_workspace_bytes(config, M, N, K)
    full = L.repops_gemm_i8_operand_workspace_bytes(config, M, N, K, b.data_ptr(), b.stride(0))
    assert full == short + (N * K if config == 1 and offset else 0)
    if config == 1:
        assert short == 5 * M * K * 2                     # five copies of the tokens (250 KB), nothing of the weights
    stream = torch.cuda.current_stream().cuda_stream
    for size in {short, full}:
        ws = torch.full((size + 256,), 99, dtype=torch.uint8, device=DEV)
        out = torch.zeros(M, N, device=DEV)
        for _ in range(2):
            rc = L.repops_gemm_i8(config, M, N, K, a.data_ptr(), K, sa.data_ptr(), b.data_ptr(), b.stride(0),
                                  sb.data_ptr(), None, out.data_ptr(), rp.TYPE_F32, N, ws.data_ptr() if size else None,
                                  size, stream)
            assert rc == 0
        assert torch.equal(out, want) and (ws[size:] == 99).all()


def test_the_bindings_scratch_does_not_hold_aligned_weights(rp):
    M, N, K = 64, 4096, 4096
    a, b = ints((M, K), 3), ints((N, K), 4)
    sa, sb, out = torch.ones(M, device=DEV), torch.ones(N, device=DEV), torch.empty(M, N, device=DEV)
    assert rp.gemm_i8_auto_config(M, N, K) == 1
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    rp.gemm_i8(a, b.t(), sa, sb, out=out)
    assert torch.cuda.max_memory_allocated() - before < 4 << 20


@pytest.mark.parametrize("config", [-1, 0, 1, 2])
def test_empty_sums_of_many_tokens(rp, config):
    M = 65535 * 64 + 77
    a, b = torch.empty(M, 0, dtype=torch.int8, device=DEV), torch.empty(2, 0, dtype=torch.int8, device=DEV)
    bias = torch.tensor([3.0, -4.0], device=DEV)
    y = rp.gemm_i8(a, b.t(), torch.ones(M, device=DEV), torch.ones(2, device=DEV), bias=bias, config=config)
    assert torch.equal(y, bias.expand(M, 2))


@pytest.mark.parametrize("K", [16, 21])
def test_few_row_kernel_with_many_tokens(rp, K):
    M, N = 65535 * 64 + 77, 2
    a, b = ints((M, K), 5), ints((N, K), 6)
    sa = torch.rand(M, device=DEV) + 0.5
    sb = torch.rand(N, device=DEV) + 0.5
    y = rp.gemm_i8(a, b.t(), sa, sb, config=0)
    want = (a.double() @ b.double().t()).float() * sa[:, None] * sb
    assert torch.equal(y, want)
    assert torch.equal(rp.gemm_i8(a, b.t(), sa, sb), want)


@pytest.mark.parametrize("offset", [0, 3])
def test_scratch_from_the_pool_also_within_a_captured_graph(rp, offset):
    """A raw stream handle takes all scratch from the library's pool; a caller's
    that holds the tokens alone only the copy of unaligned weights."""
    M, N, K = 40, 300, 640
    L = rp.load()
    a, b = ints((M, K), 7), ints((N, K + 16), 8)[:, offset:offset + K]
    sa, sb = torch.rand(M, device=DEV) + 0.5, torch.rand(N, device=DEV) + 0.5
    want = rp.gemm_i8(a, b.t(), sa, sb, config=0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for config in (1, 2):
        out = torch.zeros_like(want)
        torch.cuda.synchronize()
        rp.gemm_i8(a, b.t(), sa, sb, out=out, config=config, stream=side.cuda_stream)
        side.synchronize()
        assert torch.equal(out, want)
    size = L.repops_gemm_i8_workspace_bytes(1, M, N, K)
    graphs = []
    for with_ws in (True, False):
        out, ws = torch.zeros_like(want), torch.empty(size, dtype=torch.uint8, device=DEV)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            rc = L.repops_gemm_i8(1, M, N, K, a.data_ptr(), K, sa.data_ptr(), b.data_ptr(), b.stride(0), sb.data_ptr(), None,
                                  out.data_ptr(), rp.TYPE_F32, N, ws.data_ptr() if with_ws else None,
                                  size if with_ws else 0, torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        graphs.append((gr, out, ws))
    for _ in range(3):
        for gr, out, _ in graphs:
            out.zero_()
            gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, out, _ in graphs)
