"""The 8-bit product with scratch of exactly the size asked for, whatever the
weights' alignment."""
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
