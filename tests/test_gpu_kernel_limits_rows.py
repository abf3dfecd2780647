"""The row operators and the rolling hash at two sizes from two host threads at once
(see test_gpu_kernel_limits_threads.py)."""
import pytest
import torch

from test_gpu_kernel_limits_threads import DEV, check, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op", ["softmax", "softmax_causal", "rmsnorm", "rmsnorm_vec", "layernorm_vec", "rmsnorm_backward", "softmax_backward",
                                "edge", "rolling"])
def test_row_operators_of_two_lengths(rp, monkeypatch, op):
    """Unaligned rows of 37 columns and of 390001 (12 bytes and 50 KB of shared memory),
    causal rows of 64 and 4096, rows whose parameters are staged beside others whose are
    not, and rolling hashes of two windows."""
    def two(make, short=37, long=390_001):
        return [make(randn(2, short)), make(randn(2, long))]

    def gain(x, off=0):
        return randn(x.shape[1] + off, seed=4)[off:]

    if op == "softmax":
        calls = two(lambda x: lambda: (rp.softmax_rows(x),))
    elif op == "softmax_causal":
        calls = two(lambda x: lambda: (rp.softmax_rows(x, causal_first=1),), short=64, long=4096)
    elif op == "rmsnorm":
        calls = two(lambda x: (lambda g: lambda: (rp.rmsnorm_rows(x, g, 1e-5),))(gain(x)))
    elif op.endswith("_vec"):
        x = randn(2, 8192)
        if op == "rmsnorm_vec":
            calls = [(lambda g: lambda: (rp.rmsnorm_rows(x, g, 1e-5),))(gain(x, off)) for off in (0, 1)]
        else:
            calls = [(lambda g: lambda: (rp.layernorm_rows(x, g, g, 1e-5),))(gain(x, off)) for off in (0, 1)]
    elif op == "rmsnorm_backward":
        calls = two(lambda x: (lambda g, d: lambda: rp.rmsnorm_backward(x, g, 1e-5, d))(gain(x), randn(*x.shape, seed=5)))
    elif op == "softmax_backward":
        calls = two(lambda x: (lambda p, d: lambda: (rp.softmax_backward(p, d),))(rp.softmax_rows(x), randn(*x.shape, seed=5)))
    elif op == "edge":
        calls = two(lambda x: (lambda g, f: lambda: rp.rmsnorm_residual(x, f, g, 1e-5))(gain(x), randn(*x.shape, seed=6)),
                    short=8197)
    else:
        w = torch.randint(0, 2 ** 31 - 1, (4, 20000), generator=torch.Generator(device=DEV).manual_seed(7), device=DEV,
                          dtype=torch.int32)
        calls = [lambda n=n: (rp.rolling_hash(w, n),) for n in (2, 700)]
    check(rp, monkeypatch, calls)
