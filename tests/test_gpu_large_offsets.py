"""Elements behind the 2^32nd: log probabilities and head norms of rows far apart,
AdamW of a long tensor, each with the bits of the same values close together."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
PITCH = (1 << 27) + 8
ROWS = 36                       # the last starts behind element 2^32


def apart(t):
    """t's rows PITCH elements apart."""
    out = torch.empty((ROWS - 1) * PITCH + t.shape[1], dtype=t.dtype, device=DEV).as_strided(t.shape, (PITCH, 1))
    out.copy_(t)
    return out


def rand(cols, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(ROWS, cols, generator=g, device=DEV).to(torch.bfloat16)


def test_log_probabilities(rp):
    x, t = rand(5001, 1), torch.arange(ROWS, device=DEV) * 131 % 5001
    far = apart(x)
    a, b = rp.token_logprobs(x, t, top=4), rp.token_logprobs(far, t, top=4)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    d = torch.full((ROWS,), -0.5, device=DEV)
    want = rp.token_logprobs_backward(x, t, a.stats, d, d)
    assert torch.equal(rp.token_logprobs_backward(far, t, b.stats, d, d, out=far), want)


def test_head_norms(rp):
    x, dy = rand(5 * 64, 2), rand(5 * 64, 3)
    cos, sin = rp.rope_table(ROWS, rp.rope_frequencies(32, 9.2, DEV))
    gains = dict(q_gain=torch.rand(64, device=DEV) + 0.5, k_gain=torch.rand(64, device=DEV) + 0.5)
    far, dfar = apart(x), apart(dy)
    want = rp.head_norm_rope_backward(dy, x, 3, 2, cos, sin, **gains)
    for u, v in zip(rp.head_norm_rope_backward(dfar, far, 3, 2, cos, sin, dx=dfar, **gains), want):
        assert torch.equal(u, v)
    y = rp.head_norm_rope(x, 3, 2, cos, sin, **gains)
    assert torch.equal(rp.head_norm_rope(far, 3, 2, cos, sin, out=far, **gains), y)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(rp, bits):
    """The elements from the 2^32nd on: a dither counts elements in 32 bits, so they
    are rounded as a tensor of their own."""
    start, tail = 1 << 32, 5003
    g = torch.Generator(device=DEV).manual_seed(4)

    def pair(values):
        big = torch.zeros(start + tail, dtype=values.dtype, device=DEV)
        big[start:] = values
        return big, values

    theta, small = pair(torch.randn(tail, generator=g, device=DEV))
    grad, sgrad = pair(torch.randn(tail, generator=g, device=DEV).to(torch.bfloat16))
    state, sstate = (rp.adamw_state([t], bits=bits) for t in (theta, small))
    for t, dx, s in ((theta, grad, state), (small, sgrad, sstate)):
        for step in (1, 2):
            rp.adamw([t], [dx], step=step, lr=1e-2, weight_decay=0.1, seed=9, **s)
    assert torch.equal(theta[-tail:], small)
    assert not theta[:start:65537].any()
    for k in state:
        assert torch.equal(state[k][0][-sstate[k][0].numel():], sstate[k][0]), k
