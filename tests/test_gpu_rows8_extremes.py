"""Rows in 8 bits at the ends of their range: the largest binary32 value, groups
whose largest magnitude is below the scale's floor, rows without a column, and
gradients of no rows on a stream of their own."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
MOST = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("cols", [512, 511])
def test_the_largest_value_comes_back_finite(rp, group, cols):
    """Every finite value within scale * (1/2 + 2^-14): fl(MOST / 127) rounds up, so
    that 127 times it is an infinity; the scale is then the value below."""
    x = torch.ones(6, cols, device=DEV)
    x[0, 3] = MOST
    x[1, 500] = -MOST
    x[2] = MOST
    x[3, 40] = torch.nextafter(torch.tensor(MOST), torch.tensor(0.0))
    x[4, ::2] = MOST / 2
    x[4, 1::2] = -MOST
    x[5] = torch.linspace(-MOST / 2, MOST / 2, cols, device=DEV) * 2
    q, s = rp.quantize_rows(x, group=group)
    v = rp.dequantize_rows(q, s, group=group)
    assert torch.isfinite(s).all() and torch.isfinite(v).all()
    width = group or cols
    bound = s.double().repeat_interleave(width, 1)[:, :cols] * (0.5 + 2.0 ** -14)
    assert ((v.double() - x.double()).abs() <= bound).all()
    assert int(q[0, 3]) == 127 and int(q[1, 500]) == -127 and bool((q[2] == 127).all())
    # only that value's scale leaves fl(amax / 127)
    a = x.abs()
    a = torch.nn.functional.pad(a, (0, -cols % width)).view(6, -1, width).amax(2).cpu().numpy()
    want = a / np.float32(127)
    want[a == np.float32(MOST)] = np.nextafter(np.float32(MOST) / np.float32(127), np.float32(0))
    assert np.array_equal(s.cpu().numpy().view(np.uint32), want.view(np.uint32))


@pytest.mark.parametrize("group", [0, 32])
def test_groups_below_the_floor_are_whole_parts_of_it(rp, group):
    """amax < 2^-100 takes the floor's scale fl(2^-100 / 127), and the values their
    whole numbers of it: not all of them zeros."""
    x = torch.zeros(4, 64, device=DEV)
    x[0, 0], x[0, 40] = 2.0 ** -101, -2.0 ** -101
    x[1, 0], x[1, 40] = 2.0 ** -107, 2.0 ** -106
    x[2, 0], x[2, 40] = 2.0 ** -108, 2.0 ** -149
    q, s = rp.quantize_rows(x, group=group)
    assert (s == np.float32(2.0 ** -100) / np.float32(127)).all()
    assert q[0, [0, 40]].tolist() == [64, -64]          # 63.5, ties to even
    assert q[1, [0, 40]].tolist() == [1, 2]             # 127/128 and 127/64
    assert q[2:].abs().max() == 0                       # 127/256 < 1/2
    assert q.ne(0).sum() == 4


def test_rows_without_columns_have_the_floor_as_their_scale(rp):
    """group 0 keeps a scale a row, also of rows without a column: the maximum of
    nothing is 0.  It reaches gemm_i8, whose empty sums it must not spoil."""
    s = torch.full((5, 1), float("nan"), device=DEV)
    q, got = rp.quantize_rows(torch.empty(5, 0, device=DEV), scale=s)
    assert got is s and (s == np.float32(2.0 ** -100) / np.float32(127)).all()
    w, ws = rp.quantize_rows(torch.empty(3, 0, device=DEV))
    assert q.shape == (5, 0) and (rp.gemm_i8(q, w.t(), s.view(-1), ws.view(-1)) == 0).all()


def test_gradients_of_no_rows_are_zeroed_on_the_stream_of_the_call(rp):
    """Without rows a gain's gradient is +0 (an empty column sum), written where the
    call runs: not behind work queued on the current stream."""
    cols, side = 40, torch.cuda.Stream()
    e = torch.empty(0, cols, device=DEV)
    gain = torch.ones(cols, device=DEV)
    for handle in (side, side.cuda_stream):
        dg, dpre, dpost = (torch.full((cols,), 7.0, device=DEV) for _ in range(3))
        dgate = torch.full((3, cols + 2), 7.0, device=DEV)
        torch.cuda.synchronize()
        torch.cuda._sleep(400_000_000)                   # a fifth of a second on the current stream
        rp.rmsnorm_backward_i8(e.to(torch.int8), torch.empty(0, 1, device=DEV), gain, 1e-5, e, group=0, dgamma=dg,
                               stream=handle)
        rp.rmsnorm_residual_backward(e, e, e, e, gain, post_gain=gain, gate=torch.ones(3, cols, device=DEV), dpre=dpre,
                                     dpost=dpost, dgate=dgate[:, :cols], stream=handle)
        with torch.cuda.stream(side):
            got = torch.cat([dg, dpre, dpost, dgate.view(-1)]).cpu()
        torch.cuda.synchronize()
        assert (got[:3 * cols] == 0).all()
        assert (got[3 * cols:].view(3, -1)[:, :cols] == 0).all() and (got[3 * cols:].view(3, -1)[:, cols:] == 7).all()
    with pytest.raises(ValueError):                      # the arguments are looked at without rows too
        rp.rmsnorm_backward_i8(e.to(torch.int8), torch.empty(0, 1, device=DEV), gain, 1e-5, e, group=0, dgamma=gain[1:])
    with pytest.raises(ValueError):
        rp.rmsnorm_residual_backward(e, e, e, e, gain, dpre=gain[1:])
