"""Scratch that the binding takes from PyTorch's allocator for a call on a stream
of its own."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_scratch_is_not_memory_of_another_streams_work(rp):
    """Scratch for a call on another stream comes from that stream's own memory: a
    block that calls on the current stream may still be reading is not handed to
    it, nor the other way round."""
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    n = 3 << 20
    torch.cuda.synchronize()
    torch.cuda.empty_cache()

    def where(stream):
        ws = rp._workspace(n, torch.device(DEV), stream)
        return ws.data_ptr()                              # and free it again

    on_here = where(None)
    on_side = where(side)
    assert on_side != on_here
    assert where(here) == on_here and where(side) == on_side
    assert where(None) == on_here
    assert rp._workspace(n, torch.device(DEV), side.cuda_stream) is None


def test_calls_on_two_streams_at_once(rp):
    """Products whose tokens are widened in scratch, queued on two streams in turn
    without a wait between them, beside the GEMM and the Merkle root that take
    theirs the same way."""
    g = torch.Generator(device=DEV).manual_seed(1)
    M, N, K = 96, 640, 1024
    sets = []
    for _ in range(2):
        a = torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
        b = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
        sa, sb = torch.rand(M, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV)
        x = torch.randn(1601, 1601, generator=g, device=DEV)
        sets.append((a, b, sa, sb, rp.gemm_i8(a, b.t(), sa, sb, config=0), x, rp.gemm(x, x, config=0)))
    roots = [rp.merkle_sha256(s[5]) for s in sets]
    side = torch.cuda.Stream()
    outs = [[torch.empty_like(s[4]) for _ in range(16)] for s in sets]
    prods = [[torch.empty_like(s[6]) for _ in range(2)] for s in sets]
    torch.cuda.synchronize()
    for i in range(16):
        for st, (a, b, sa, sb, *_), out in zip((None, side), sets, outs):
            rp.gemm_i8(a, b.t(), sa, sb, out=out[i], config=1 + i % 2, stream=st)
    for i in range(2):
        for st, s, p in zip((None, side), sets, prods):
            rp.gemm(s[5], s[5], out=p[i], stream=st)
    torch.cuda.synchronize()
    for s, out, p, root in zip(sets, outs, prods, roots):
        assert all(torch.equal(o, s[4]) for o in out) and all(torch.equal(o, s[6]) for o in p)
        assert torch.equal(rp.merkle_sha256(s[5]), root)
