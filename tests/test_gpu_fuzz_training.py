"""Seeded random cases of the log probabilities, the head norms with rotations and
AdamW: sizes spread over their logarithm, odd widths, pitches, offsets, storage
types, masked and empty rows, missing operands and in-place outputs, each bit for
bit against the step-by-step statements in NumPy."""
import random

import numpy as np
import pytest
import torch

import adamw_ref
import headnorm_ref
import logprobs_ref
from test_gpu_adamw import problem as adam_problem, restored
from test_gpu_headnorm import by_head, gains, host, narrowed, problem as head_problem, same
from test_gpu_logprobs import DEV, DT, check, logits

pytestmark = pytest.mark.gpu

KINDS = ["f32", "f16", "bf16"]


def log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


@pytest.mark.parametrize("seed", range(60))
def test_log_probabilities(rp, seed):
    rng = random.Random(seed)
    kind, cols = rng.choice(KINDS), log(rng, 1, 30000)
    rows = log(rng, 1, max(1, min(200, 300000 // cols)))
    T = rng.choice([1.0, 0.5, 0.9, 1.7, 30.0])
    x = logits(rows, cols, kind, seed, rng.choice([0, 0, 1, 3, 8]), rng.choice([0, 0, 1, 2, 5]), rng.choice([0.1, 3.0, 20.0]))
    for _ in range(rng.randint(0, 3)):                      # columns, a row's part, a whole row that is impossible
        a, b = sorted(rng.randint(0, cols) for _ in range(2))
        x[rng.randint(0, rows - 1) if rng.random() < 0.5 else slice(None), a:b] = -np.inf
    if rng.random() < 0.3:
        x[rng.randint(0, rows - 1)] = -np.inf
    if rng.random() < 0.2:
        x[rng.randint(0, rows - 1), rng.randint(0, cols - 1)] = rng.choice([np.nan, np.inf, torch.finfo(DT[kind]).min])
    t = torch.randint(-1, cols, (rows,), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)
    if rng.random() < 0.1:
        t[rng.randint(0, rows - 1)] = cols
    t = None if rng.random() < 0.1 else t
    got = check(rp, x, t, T, min(cols, rng.choice([0, 1, 2, 7, 31, 32])))
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    dl, de = (torch.randn(rows, generator=g, device=DEV) for _ in range(2))
    if t is None:
        dl = None
    elif rng.random() < 0.5:
        de = None
    out = rng.choice([None, "x", "pitched"])
    want = logprobs_ref.backward(host(x), None if t is None else host(t).astype(np.int64), host(got.stats),
                                 None if dl is None else host(dl), None if de is None else host(de), T)
    if out == "pitched":
        out = logits(rows, cols, kind, seed, rng.choice([0, 1, 4]), rng.choice([0, 1, 3]))
    elif out == "x":
        out = x
    d = rp.token_logprobs_backward(x, t, got.stats, dl, de, temperature=T, out=out)
    assert (out is None or d is out) and same(host(d), host(torch.from_numpy(want).to(DT[kind])))


@pytest.mark.parametrize("seed", range(60))
def test_heads(rp, seed):
    rng = random.Random(seed)
    kind, layout = rng.choice(KINDS), rng.choice(["adjacent", "halves"])
    dim = rng.choice([64, 80, 128, 4 * rng.randint(1, 128), log(rng, 1, 512)])
    pairs = rng.choice([dim // 2, dim // 4, rng.randint(0, dim // 2), 0])
    q, k = rng.randint(0, 6), rng.randint(0, 3)
    q = q or int(k == 0)
    rows = log(rng, 1, max(1, min(600, 200000 // ((q + k) * dim))))
    o = head_problem(rows, q, k, dim, pairs, kind, seed, rng.choice([0, 0, 1, 4, 8]), rng.choice([0, 0, 1, 4]))
    pos, where = o["pos"].cpu().numpy(), dict(positions=o["pos"].int() if rng.random() < 0.5 else o["pos"])
    if rng.random() < 0.5:
        first, period = rng.randint(0, 9), rng.randint(1, 40)
        pos, where = first + np.arange(rows) % period, dict(first=first, period=period)
    elif rng.random() < 0.3:
        where["positions"][0] = pos[0] = 50 + rng.randint(0, 5)         # past the table
    cos, sin = (None if o[n] is None else host(o[n]) for n in ("cos", "sin"))
    kw = dict(eps=rng.choice([1e-6, 1e-3]), layout=layout, **where)
    x, live = by_head(o["x"], dim), (pos >= 0)[:, None]
    g = gains(o, q, k)
    gain = dict(q_gain=o["q_gain"], k_gain=o["k_gain"])
    want = narrowed(headnorm_ref.forward(x, g, kw["eps"], cos, sin, pos, layout), kind).reshape(rows, -1)
    got = rp.head_norm_rope(o["x"], q, k, o["cos"], o["sin"], **gain, **kw)
    assert same(host(got), np.where(live, want, 0))
    back = rng.random() < 0.5
    want = narrowed(headnorm_ref.forward(x, None, 0.0, cos, sin, pos, layout, back), kind).reshape(rows, -1)
    y = o["x"].clone(memory_format=torch.preserve_format)
    rp.head_norm_rope(y, q, k, o["cos"], o["sin"], inverse=back, out=y, **kw)
    assert same(host(y), np.where(live, want, host(o["x"])))
    dx, terms = headnorm_ref.backward(by_head(o["dy"], dim), x, g, kw["eps"], cos, sin, pos, layout)
    dy = o["dy"].clone(memory_format=torch.preserve_format)
    out = dy if rng.random() < 0.5 else None
    d, dq, dk = rp.head_norm_rope_backward(dy, o["x"], q, k, o["cos"], o["sin"], dx=out, **gain, **kw)
    assert same(host(d), np.where(live, narrowed(dx, kind).reshape(rows, -1), 0 if out is None else host(o["dy"])))
    for t, part in ((dq, terms[:, :q]), (dk, terms[:, q:])):
        assert (t is None) == (part.shape[1] == 0)
        if t is not None:
            assert same(host(t), headnorm_ref.colsum(part))


@pytest.mark.parametrize("seed", range(60))
def test_adamw(rp, seed):
    rng = random.Random(seed)
    bits, kind, k = rng.choice([32, 8]), rng.choice(KINDS), rng.choice([1, 1, 2, 3, 5, 8, 33])
    sizes = [rng.choice([0, log(rng, 1, 9000), 128 * rng.randint(1, 40)]) for _ in range(rng.randint(1, 12))]
    theta, grads, st = adam_problem(sizes, k, kind, 1000 * seed, rng.choice([0, 0, 1, 4]), bits)
    order = list(range(k))
    rng.shuffle(order)
    hyper = dict(betas=(rng.choice([0.0, 0.9]), rng.choice([0.0, 0.95, 0.999])), eps=rng.choice([1e-8, 1e-4]))
    step, lr, key = rng.choice([1, 2, 1000, 1 << 33]), rng.choice([0.0, 1e-3]), rng.choice([0, 7, (1 << 32) - 1])
    decay = [rng.choice([0.0, 0.1]) for _ in sizes]
    scale = torch.tensor([rng.choice([0.37, 1.0])], device=DEV) if rng.random() < 0.4 else None
    was = [(host(t), [host(grads[c][i]) for c in order]) +
           (restored(st, i) if bits == 8 else (host(st["m"][i]), host(st["v"][i]))) for i, t in enumerate(theta)]
    how = dict(step=step, lr=lr, seed=key)
    if rng.random() < 0.4:
        how = dict(scalars=rp.adamw_scalars(step, lr, hyper["betas"], key).to(DEV))
    words = rp.adamw_scalars(step, lr, hyper["betas"], key).numpy()
    sc = tuple(words[:3].view(np.float32)) + (int(words[3:].view(np.uint32)[0]),)
    rp.adamw(theta, grads, **st, weight_decay=decay, order=order, grad_scale=scale, **how, **hyper)
    for i, (t, g, m, v) in enumerate(was):
        want = adamw_ref.step(t, g, m, v * v if bits == 8 else v, sc, decay[i], hyper["betas"], hyper["eps"],
                              None if scale is None else float(scale))
        assert same(host(theta[i]), want[0])
        if bits == 32:
            assert same(host(st["m"][i]), want[1]) and same(host(st["v"][i]), want[2])
        else:
            dm, dr = adamw_ref.dither(sizes[i], sc[3], i)
            got = restored(st, i)
            assert same(got[0], adamw_ref.coded(want[1], False, dm)[0])
            assert same(got[1], adamw_ref.coded(want[3], True, dr)[0])
            m, v = rp.adamw_moments(*(st[n][i] for n in ("m", "v", "m_scales", "v_scales")))
            assert same(host(m), got[0]) and same(host(v), got[1] * got[1])
