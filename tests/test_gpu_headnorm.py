"""Norms of query and key heads with the rotation on the GPU: bit for bit against the
step-by-step definition and against the library's separate operators, and against
binary64; widths from one column to 512, odd ones, part of a head rotated, both
layouts, every storage type, pitches and misaligned bases, positions of all kinds,
in place, streams, graphs and refusals."""
import math

import numpy as np
import pytest
import torch

import headnorm_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32 = np.float32
EPS = 1e-6
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
# dim, pairs
SHAPES = [(64, 32), (128, 64), (80, 16), (96, 48), (32, 16), (256, 32), (512, 256), (1, 0), (2, 1), (7, 3), (33, 16),
          (66, 33), (100, 6), (64, 0), (192, 64), (36, 18)]


def host(t):
    return t.detach().float().cpu().numpy()


def same(a, b):
    a, b = np.asarray(a, F32), np.asarray(b, F32)
    both = np.isnan(a) & np.isnan(b)
    return a.shape == b.shape and np.array_equal(np.where(both, 0, a).view(np.uint32), np.where(both, 0, b).view(np.uint32))


def randn(shape, seed, sd=1.0):
    return torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * sd


def rows_of(rows, width, kind, seed, pad=0, off=0, sd=1.5):
    flat = randn(rows * (width + pad) + off + 1, seed, sd).to(DT[kind])
    return flat.as_strided((rows, width), (width + pad, 1), off)


def tables(positions, pairs):
    if pairs == 0:
        return None, None
    f = torch.exp(torch.arange(pairs, device=DEV, dtype=torch.float64) * (-math.log(500000.0) / pairs)).float()
    a = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * f.double()
    return a.cos().float(), a.sin().float()


def problem(rows, q, k, dim, pairs, kind, seed, pad=0, off=0, padded=True):
    width = (q + k) * dim
    p = torch.randint(0, 50, (rows,), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)
    if padded and rows > 3:
        p[2] = -1
        p[-1] = -7
    cos, sin = tables(50, pairs)
    return dict(x=rows_of(rows, width, kind, seed, pad, off), dy=rows_of(rows, width, kind, seed + 1, pad, off, 1e-2),
                cos=cos, sin=sin, pos=p, q_gain=1 + 0.1 * randn((dim,), seed + 2), k_gain=1 + 0.1 * randn((dim,), seed + 3))


def by_head(t, dim):
    return host(t).reshape(t.shape[0], -1, dim)


def gains(o, q, k):
    return np.concatenate([np.tile(host(o["q_gain"]), (q, 1)), np.tile(host(o["k_gain"]), (k, 1))])


def arrays(o):
    return [None if o[n] is None else host(o[n]) for n in ("cos", "sin")] + [o["pos"].cpu().numpy()]


def narrowed(a, kind):
    return host(torch.from_numpy(np.ascontiguousarray(a)).to(DT[kind]))


@pytest.mark.parametrize("dim,pairs", SHAPES)
@pytest.mark.parametrize("layout", ["adjacent", "halves"])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_forward(rp, dim, pairs, layout, kind):
    for rows, q, k, pad, off in ((1, 1, 0, 0, 0), (5, 3, 1, 0, 0), (9, 4, 2, 3, 1), (70, 2, 2, 8, 4), (6, 0, 2, 4, 0)):
        o = problem(rows, q, k, dim, pairs, kind, dim + rows, pad, off)
        x, (cos, sin, pos) = by_head(o["x"], dim), arrays(o)
        live = (pos >= 0)[:, None]
        for normed in (True, False):
            g = gains(o, q, k) if normed else None
            kw = dict(q_gain=o["q_gain"], k_gain=o["k_gain"]) if normed else {}
            want = narrowed(ref.forward(x, g, EPS, cos, sin, pos, layout), kind).reshape(rows, -1)
            buf = torch.full((rows * ((q + k) * dim + pad) + off + 1,), 7.0, dtype=DT[kind], device=DEV)
            out = buf.as_strided(o["x"].shape, o["x"].stride(), off)
            for p in (o["pos"], o["pos"].int()):
                rp.head_norm_rope(o["x"], q, k, o["cos"], o["sin"], eps=EPS, layout=layout, positions=p, out=out, **kw)
                assert same(host(out), np.where(live, want, 7))
            rest = buf.clone()
            rest.as_strided(out.shape, out.stride(), off).fill_(7.0)
            assert (rest == 7).all()                        # nothing between or behind its rows
            y = o["x"].clone(memory_format=torch.preserve_format)
            rp.head_norm_rope(y, q, k, o["cos"], o["sin"], eps=EPS, layout=layout, positions=o["pos"], out=y, **kw)
            assert same(host(y), np.where(live, want, host(o["x"])))
            val, bound = ref.forward64(x, g, EPS, cos, sin, pos, layout)
            err = np.abs(host(out).reshape(val.shape) - val)[pos >= 0]
            assert (err <= (bound + np.abs(val) * HALF[kind] * 1.01 + TINY[kind])[pos >= 0]).all()
            if not normed and pairs:
                want = narrowed(ref.forward(x, None, EPS, cos, sin, pos, layout, True), kind).reshape(rows, -1)
                rp.head_norm_rope(o["x"], q, k, o["cos"], o["sin"], layout=layout, positions=o["pos"], out=out,
                                  inverse=True)
                assert same(host(out), np.where(live, want, 7))


@pytest.mark.parametrize("dim,pairs", SHAPES)
@pytest.mark.parametrize("layout", ["adjacent", "halves"])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_backward(rp, dim, pairs, layout, kind):
    for rows, q, k, pad, off in ((1, 1, 0, 0, 0), (5, 3, 1, 0, 0), (9, 4, 2, 3, 1), (70, 5, 2, 8, 4), (6, 0, 2, 4, 0)):
        o = problem(rows, q, k, dim, pairs, kind, dim + 3 * rows, pad, off)
        x, dy, (cos, sin, pos) = by_head(o["x"], dim), by_head(o["dy"], dim), arrays(o)
        live = (pos >= 0)[:, None]
        args = (dy, x, gains(o, q, k), EPS, cos, sin, pos, layout)
        dx, terms = ref.backward(*args)
        (vx, bx), (vt, bt) = ref.backward64(*args)
        want = narrowed(dx, kind).reshape(rows, -1)
        out = torch.full_like(o["x"], 7.0)
        got = rp.head_norm_rope_backward(o["dy"], o["x"], q, k, o["cos"], o["sin"], q_gain=o["q_gain"],
                                         k_gain=o["k_gain"], eps=EPS, layout=layout, positions=o["pos"], dx=out)
        assert got[0] is out and same(host(out), np.where(live, want, 7))
        err = np.abs(host(out).reshape(vx.shape) - vx)[pos >= 0]
        assert (err <= (bx + np.abs(vx) * HALF[kind] * 1.01 + TINY[kind])[pos >= 0]).all()
        for d, part in ((got[1], slice(0, q)), (got[2], slice(q, q + k))):
            n = part.stop - part.start
            assert (d is None) == (n == 0)
            if n:
                assert same(host(d), ref.colsum(terms[:, part]))
                t, b = vt[:, part].reshape(-1, dim), bt[:, part].reshape(-1, dim)
                # a sum of n terms adds at most 32 half steps a level of the tree
                levels = max(1, math.ceil(math.log(max(len(t), 2), 32)))
                assert (np.abs(host(d) - t.sum(0)) <= b.sum(0) + np.abs(t).sum(0) * 32 * levels * ref.U).all()
        y = o["dy"].clone(memory_format=torch.preserve_format)
        rp.head_norm_rope_backward(y, o["x"], q, k, o["cos"], o["sin"], q_gain=o["q_gain"], k_gain=o["k_gain"], eps=EPS,
                                   layout=layout, positions=o["pos"], dx=y)
        assert same(host(y), np.where(live, want, host(o["dy"])))


@pytest.mark.parametrize("rows,q,k,dim", [(64, 8, 2, 64), (300, 6, 3, 128), (33, 4, 1, 40)])
def test_equals_the_separate_operators(rp, rows, q, k, dim):
    """rmsnorm_rows on the heads, then rope; their backward operators and colsum."""
    o = problem(rows, q, k, dim, dim // 2, "f32", rows, padded=False)
    cos, sin = rp.rope_table(rows, rp.rope_frequencies(dim // 2, math.log(500000.0)))
    x = o["x"].contiguous()
    y = rp.head_norm_rope(x, q, k, cos, sin, q_gain=o["q_gain"], k_gain=o["k_gain"], eps=EPS)
    parts = []
    for lo, n, g in ((0, q, "q_gain"), (q, k, "k_gain")):
        h = x[:, lo * dim:(lo + n) * dim].reshape(-1, dim).contiguous()
        parts.append(rp.rmsnorm_rows(h, o[g], EPS).view(rows, n * dim))
    want = rp.rope(torch.cat(parts, 1).contiguous(), q + k, cos, sin)
    assert torch.equal(y, want)
    dx, dq, dk = rp.head_norm_rope_backward(o["dy"], x, q, k, cos, sin, q_gain=o["q_gain"], k_gain=o["k_gain"], eps=EPS)
    g = rp.rope(o["dy"].contiguous().clone(), q + k, cos, sin, inverse=True)
    assert torch.equal(g, rp.head_norm_rope(o["dy"], q, k, cos, sin, inverse=True))
    for lo, n, name, d in ((0, q, "q_gain", dq), (q, k, "k_gain", dk)):
        cut = lambda t: t[:, lo * dim:(lo + n) * dim].reshape(-1, dim).contiguous()
        hx, t = rp.rmsnorm_backward(cut(x), o[name], EPS, cut(g))
        assert torch.equal(cut(dx), hx) and torch.equal(d, rp.colsum(t))


def test_long_sums(rp):
    """More than 1024 and more than 32768 runs of a gain's sum: the further levels."""
    for rows, q, k, dim in ((5000, 8, 8, 8), (34000, 33, 1, 4), (36000, 33, 31, 2)):
        o = problem(rows, q, k, dim, dim // 2, "f32", 5, padded=False)
        d = rp.head_norm_rope_backward(o["dy"], o["x"], q, k, o["cos"], o["sin"], q_gain=o["q_gain"], k_gain=o["k_gain"],
                                       eps=EPS, positions=o["pos"])
        cos, sin, pos = arrays(o)
        _, terms = ref.backward(by_head(o["dy"], dim), by_head(o["x"], dim), gains(o, q, k), EPS, cos, sin, pos, "adjacent")
        assert same(host(d[1]), ref.colsum(terms[:, :q])) and same(host(d[2]), ref.colsum(terms[:, q:]))


def test_positions(rp):
    """By first and period, far ones, one past the table (NaN where it rotates), a
    batch of padding alone."""
    o = problem(12, 2, 1, 64, 16, "f32", 9)
    kw = dict(q_gain=o["q_gain"], k_gain=o["k_gain"], eps=EPS)
    a = rp.head_norm_rope(o["x"], 2, 1, o["cos"], o["sin"], first=3, period=5, **kw)
    p = 3 + torch.arange(12, device=DEV) % 5
    assert torch.equal(a, rp.head_norm_rope(o["x"], 2, 1, o["cos"], o["sin"], positions=p, **kw))
    p[4] = 50
    p[5] = 1 << 40
    b = rp.head_norm_rope(o["x"], 2, 1, o["cos"], o["sin"], positions=p, **kw).view(12, 3, 64)
    assert torch.isnan(b[4:6, :, :32]).all() and torch.isfinite(b[4:6, :, 32:]).all()
    rest = [r for r in range(12) if r not in (4, 5)]
    assert torch.equal(b[rest], a.view(12, 3, 64)[rest])
    none = torch.full((12,), -1, device=DEV)
    out = torch.full_like(o["x"], 3.0)
    rp.head_norm_rope(o["x"], 2, 1, o["cos"], o["sin"], positions=none, out=out, **kw)
    assert (out == 3).all()
    out, dq, dk = rp.head_norm_rope_backward(o["dy"], o["x"], 2, 1, o["cos"], o["sin"], positions=none, dx=out, **kw)
    assert (out == 3).all() and (dq == 0).all() and (dk == 0).all()
    # padding adds nothing whatever it holds, eps 0 and NaN included
    x, dy = o["x"].clone(), o["dy"].clone()
    x[2], dy[2] = 0.0, float("nan")
    x[11] = float("nan")
    d = rp.head_norm_rope_backward(dy, x, 2, 1, o["cos"], o["sin"], positions=o["pos"], q_gain=o["q_gain"],
                                   k_gain=o["k_gain"], eps=0.0)
    keep = [r for r in range(12) if r not in (2, 11)]
    assert torch.isfinite(d[1]).all() and torch.isfinite(d[0][keep]).all()


def test_scaled_frequencies(rp):
    f = rp.rope_frequencies(32, math.log(500000.0))
    f64 = f.double().cpu().numpy()
    assert np.array_equal(host(rp.rope_frequencies(32, math.log(500000.0), factor=4.0)), (f64 / 4).astype(F32))
    got = host(rp.rope_frequencies(32, math.log(500000.0), factor=8.0, original=8192, low=1.0, high=4.0))
    turns = 8192 * f64 / (2 * math.pi)
    w = np.clip((turns - 1) / 3, 0, 1)
    want = f64 / 8 + w * (f64 - f64 / 8)
    assert (np.abs(got - want) <= want * (2.0 ** -24 + 2.0 ** -50)).all()
    assert (got[turns >= 4] == host(f)[turns >= 4]).all() and (w > 0).any() and (w < 1).any()
    for bad in (dict(factor=0.0), dict(factor=-1.0), dict(factor=2.0, original=-1), dict(factor=2.0, original=8, low=4, high=1)):
        with pytest.raises(rp.RepopsError):
            rp.rope_frequencies(32, math.log(500000.0), **bad)


def test_gradient_is_the_difference_quotient(rp):
    """sum(w * y) of the library's forward at x +- h: its error is h^2 / 6 of the third
    derivative, under 60 / rms^3 of weights of 1, and the forward's 2^-21 of values of
    up to 5 over h."""
    rows, q, k, dim, h = 3, 2, 1, 32, 2.0 ** -7
    o = problem(rows, q, k, dim, 12, "f32", 21, padded=False)
    x = torch.round(o["x"] * 64) / 64 + 2.0                 # rms about 2.5
    w = torch.where(o["dy"] > 0, 1.0, -1.0)
    kw = dict(positions=o["pos"], eps=EPS, layout="halves")
    dx, dq, dk = rp.head_norm_rope_backward(w, x, q, k, o["cos"], o["sin"], q_gain=o["q_gain"], k_gain=o["k_gain"], **kw)
    loss = lambda xx, qg, kg: (rp.head_norm_rope(xx, q, k, o["cos"], o["sin"], q_gain=qg, k_gain=kg, **kw).double() *
                               w.double()).sum(1)
    tol = h * h * 10 + dim * 5 * 2.0 ** -21 / h
    for j in (0, 5, 31, 32, 64, 95):
        d = torch.zeros_like(x)
        d[:, j] = h
        up, dn = (loss(x + s * d, o["q_gain"], o["k_gain"]) for s in (1, -1))
        assert ((up - dn) / (2 * h) - dx[:, j]).abs().max() <= tol
    for j in (0, 13, 31):
        d = torch.zeros(dim, device=DEV)
        d[j] = h
        for grad, s in ((dq, (1, 0)), (dk, (0, 1))):
            up, dn = (loss(x, o["q_gain"] + t * s[0] * d, o["k_gain"] + t * s[1] * d).sum() for t in (1, -1))
            assert abs((up - dn) / (2 * h) - grad[j]) <= rows * q * tol


def test_streams_graphs_and_no_rows(rp):
    o = problem(200, 8, 2, 64, 32, "bf16", 4)
    kw = dict(q_gain=o["q_gain"], k_gain=o["k_gain"], eps=EPS, positions=o["pos"], layout="halves")
    a = rp.head_norm_rope(o["x"], 8, 2, o["cos"], o["sin"], **kw)
    b = rp.head_norm_rope_backward(o["dy"], o["x"], 8, 2, o["cos"], o["sin"], **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a2 = torch.zeros_like(a)
    d2 = torch.zeros_like(b[0])
    s.wait_stream(torch.cuda.current_stream())
    rp.head_norm_rope(o["x"], 8, 2, o["cos"], o["sin"], out=a2, stream=s, **kw)
    b2 = rp.head_norm_rope_backward(o["dy"], o["x"], 8, 2, o["cos"], o["sin"], dx=d2, stream=s, **kw)
    s.synchronize()
    assert torch.equal(a, a2) and all(torch.equal(p, r) for p, r in zip(b, b2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = rp.head_norm_rope(o["x"], 8, 2, o["cos"], o["sin"], **kw)
        d = rp.head_norm_rope_backward(o["dy"], o["x"], 8, 2, o["cos"], o["sin"], **kw)
    o["x"].copy_(randn(o["x"].shape, 77).bfloat16())
    graph.replay()
    e = rp.head_norm_rope_backward(o["dy"], o["x"], 8, 2, o["cos"], o["sin"], **kw)
    assert torch.equal(c, rp.head_norm_rope(o["x"], 8, 2, o["cos"], o["sin"], **kw))
    assert all(torch.equal(p, r) for p, r in zip(d, e))
    x = torch.empty(0, 10 * 64, device=DEV)
    assert rp.head_norm_rope(x, 8, 2, o["cos"], o["sin"]).shape == x.shape
    z = rp.head_norm_rope_backward(x, x.clone(), 8, 2, o["cos"], o["sin"], q_gain=o["q_gain"], k_gain=o["k_gain"])
    assert (z[1] == 0).all() and (z[2] == 0).all()


def test_refusals(rp):
    o = problem(6, 2, 1, 64, 32, "f32", 3)
    x, cos, sin = o["x"], o["cos"], o["sin"]
    g = dict(q_gain=o["q_gain"], k_gain=o["k_gain"])

    def refused(exc, *args, **kw):
        with pytest.raises(exc):
            rp.head_norm_rope(*args, **kw)

    refused(ValueError, x, 3, 2, cos, sin)                   # 192 columns are no multiple of 5 heads
    refused(ValueError, x, 2, 1, cos, None)
    refused(ValueError, x, 2, 1, cos, sin[:, :5])
    refused(ValueError, x, 2, 1, cos, sin, layout="other")
    refused(ValueError, x, 2, 1, cos, sin, q_gain=o["q_gain"][:5], k_gain=o["k_gain"])
    refused(ValueError, x, 2, 1, cos, sin, positions=o["pos"][:3])
    refused(ValueError, x, 2, 1, cos, sin, positions=o["pos"].float())
    refused(ValueError, x, 2, 1, cos, sin, positions=o["pos"].cpu())
    refused(ValueError, x.t(), 2, 1, cos, sin)
    refused(ValueError, x[:1].expand(6, 192), 2, 1, cos, sin)
    refused(ValueError, x, 2, 1, cos, sin, out=torch.empty(6, 192, device=DEV, dtype=torch.float16))
    refused(TypeError, x.double(), 2, 1, cos, sin)
    refused(rp.RepopsError, x, 2, 1, cos, sin, q_gain=o["q_gain"])                  # one gain for two kinds
    refused(rp.RepopsError, x, 2, 1, cos, sin, inverse=True, **g)
    refused(rp.RepopsError, x, 2, 1, cos.repeat(1, 2), sin.repeat(1, 2))            # 64 pairs in 64 columns
    refused(rp.RepopsError, x, 2, 1, cos, sin, first=45)                            # leaves the table
    refused(rp.RepopsError, x, 2, 1, cos, sin, first=-1)
    refused(rp.RepopsError, torch.empty(2, 513, device=DEV), 1, 0)                  # above 512 columns
    refused(rp.RepopsError, x[:5], 2, 1, cos, sin, out=x[1:])                       # over other rows
    with pytest.raises(ValueError):
        rp.head_norm_rope_backward(o["dy"], x, 2, 1, cos, sin, q_gain=o["q_gain"])
    with pytest.raises(ValueError):
        rp.head_norm_rope_backward(o["dy"][:5], x, 2, 1, cos, sin, **g)
    with pytest.raises(rp.RepopsError):
        rp.head_norm_rope_backward(o["dy"], x, 2, 1, cos, sin, dx=x, **g)           # x is read again
    with pytest.raises(rp.RepopsError):
        rp.head_norm_rope_backward(o["dy"], x, 2, 1, cos, sin, dq_gain=o["k_gain"], **g)
