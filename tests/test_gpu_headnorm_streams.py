"""Outputs that head_norm_rope and its backward make themselves, with rows left
alone, on another stream than the current one: their zeros are written in the order
of the call's stream, however far behind the current one is."""
import pytest
import torch

from test_gpu_headnorm import DEV, EPS, problem

pytestmark = pytest.mark.gpu


def busy():
    """Work on the current stream for a few hundred milliseconds: what is queued there
    behind it comes long after a call on another stream has ended."""
    a = torch.randn(8192, 8192, device=DEV)
    b = torch.empty_like(a)
    torch.cuda.synchronize()

    def go():
        for _ in range(12):
            torch.mm(a, a, out=b)

    return go


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("raw", [False, True])
def test_zeros_come_before_the_results(rp, kind, raw):
    o = problem(700, 8, 2, 64, 32, kind, 9)
    kw = dict(q_gain=o["q_gain"], k_gain=o["k_gain"], eps=EPS, positions=o["pos"], layout="halves")
    want = rp.head_norm_rope(o["x"], 8, 2, o["cos"], o["sin"], **kw)
    back = rp.head_norm_rope_backward(o["dy"], o["x"], 8, 2, o["cos"], o["sin"], **kw)
    alone = rp.head_norm_rope(o["x"], 8, 2, o["cos"], o["sin"], positions=o["pos"], inverse=True)
    left = o["pos"] < 0
    assert left.any() and all((t[left] == 0).all() and t[~left].any() for t in (want, back[0], alone))
    go = busy()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    go()
    where = s.cuda_stream if raw else s
    got = rp.head_norm_rope(o["x"], 8, 2, o["cos"], o["sin"], stream=where, **kw)
    got_back = rp.head_norm_rope_backward(o["dy"], o["x"], 8, 2, o["cos"], o["sin"], stream=where, **kw)
    got_alone = rp.head_norm_rope(o["x"], 8, 2, o["cos"], o["sin"], positions=o["pos"], inverse=True, stream=where)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got_alone, alone)
    assert all(torch.equal(p, r) for p, r in zip(got_back, back))


@pytest.mark.parametrize("handle", [0, 1, 2])
def test_the_runtimes_own_handles(rp, handle):
    """The default stream by both of its names, and a thread's own."""
    o = problem(70, 2, 1, 64, 32, "f32", 3)
    want = rp.head_norm_rope(o["x"], 2, 1, o["cos"], o["sin"], positions=o["pos"])
    go = busy()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        go()
        got = rp.head_norm_rope(o["x"], 2, 1, o["cos"], o["sin"], positions=o["pos"], stream=handle)
        assert torch.cuda.current_stream() == side
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
