"""AdamW with 8-bit moments over hundreds of steps: the statement's bits at every one
of them, and what the codes do to the moments beside those in 32 bits."""
import numpy as np
import pytest
import torch

import adamw_ref as ref
from test_gpu_adamw import DEV, host, restored, same

pytestmark = pytest.mark.gpu


def gradients(n, steps, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    size = torch.exp(torch.randn(-(-n // 128), generator=g, device=DEV)).repeat_interleave(128)[:n] * 1e-3
    for _ in range(steps):
        yield torch.randn(n, generator=g, device=DEV) * size


def test_hundreds_of_steps_are_the_statements(rp):
    n, betas = 700, (0.9, 0.999)
    theta = torch.randn(n, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV) * 0.02
    st = rp.adamw_state([theta], 8)
    t, m, r = host(theta), np.zeros(n, np.float32), np.zeros(n, np.float32)
    for step, g in enumerate(gradients(n, 200, 2), 1):
        rp.adamw([theta], [g], **st, step=step, lr=1e-3, betas=betas, seed=9)
        sc = ref.scalars(step, 1e-3, betas, 9)
        t, m, _, r = ref.step(t, [host(g)], m, r * r, sc, 0.0, betas, 1e-8)
        dm, dr = ref.dither(n, sc[3], 0)
        m, r = ref.coded(m, False, dm)[0], ref.coded(r, True, dr)[0]
        if step % 20 == 0:
            got = restored(st, 0)
            assert same(host(theta), t) and same(got[0], m) and same(got[1], r), step


@pytest.mark.parametrize("beta2,steps,most", [(0.95, 300, 1.02), (0.98, 600, 1.052)])
def test_8_bit_moments_beside_32_bit_ones(rp, beta2, steps, most):
    """A code rounds the root r to one of two neighbours, right on average, with a variance
    of at most a quarter of their distance squared; that is at most r / 16, so the mean
    of r^2 comes out at most e = 2^-10 above r^2, and never below it.  A step keeps
    beta2 of that: the sum over all elements lies between the 32-bit one and (1 - beta2)
    (1 + e) / (1 - beta2 (1 + e)) of it, which is `most`.  An element's own spread: a root's
    error shrinks by beta2 a step, variance e / (1 - beta2^2) of r^2, so that of its square
    is at most 4 e / (1 - beta2^2); the elements round independently.  The first moment's
    codes are m / 8 apart at most: variance m^2 / 256 a step, without a bias."""
    n, beta1, e = 1 << 16, 0.9, 2.0 ** -10
    theta = [torch.zeros(n, device=DEV) for _ in range(2)]
    states = [rp.adamw_state([t], b) for t, b in zip(theta, (8, 32))]
    largest = 0.0
    for step, g in enumerate(gradients(n, steps, 3), 1):
        for t, st in zip(theta, states):
            rp.adamw([t], [g], **st, step=step, lr=0.0, betas=(beta1, beta2))
        largest = torch.maximum(states[1]["m"][0].abs(), torch.as_tensor(largest, device=DEV))
    m8, v8 = rp.adamw_moments(*(states[0][k][0] for k in ("m", "v", "m_scales", "v_scales")))
    m32, v32 = states[1]["m"][0].double(), states[1]["v"][0].double()
    spread = 5 * float(v32.square().sum().sqrt() / v32.sum()) * (4 * e / (1 - beta2 ** 2)) ** 0.5
    ratio = float(v8.double().sum() / v32.sum())
    assert 1 - spread <= ratio <= most + spread, ratio
    # five standard errors, the largest |m| of the run in the place of each step's
    bound = 5 * float(largest.double().square().sum().sqrt()) * (1 / 256 / (1 - beta1 ** 2)) ** 0.5
    assert abs(float((m8.double() - m32).sum())) <= bound
