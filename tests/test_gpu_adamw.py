"""AdamW over many tensors on the GPU: bit for bit against the step-by-step
binary32 statement (moments in 32 bits and in 8), and against the formula in
binary64; sizes from none to several tiles, unaligned tensors, contributors in
every order, clipping, values that are not finite, streams, graphs and refusals."""
import numpy as np
import pytest
import torch

import adamw_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32 = np.float32
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HYPER = dict(betas=(0.9, 0.95), eps=1e-8)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(n, seed, sd=1.0, off=0):
    """n values `off` elements behind the start of their memory."""
    return (torch.randn(n + off, generator=gen(seed), device=DEV) * sd)[off:]


def host(t):
    return t.detach().float().cpu().numpy()


def same(a, b):
    a, b = np.asarray(a, F32), np.asarray(b, F32)
    both = np.isnan(a) & np.isnan(b)
    return a.shape == b.shape and np.array_equal(np.where(both, 0, a).view(np.uint32), np.where(both, 0, b).view(np.uint32))


def problem(sizes, k, kind, seed, off=0, bits=32):
    """theta, contributors' gradients and moments; `off` misaligns every tensor."""
    theta = [randn(n, seed + 7 * i, 0.02, off) for i, n in enumerate(sizes)]
    grads = [[randn(n, seed + 7 * i + 100003 * (c + 1), 1e-3, off).to(DT[kind]) for i, n in enumerate(sizes)]
             for c in range(k)]
    if off:                                     # .to() made new memory
        grads = [[torch.cat([g.new_zeros(off), g])[off:] for g in gs] for gs in grads]
    if bits == 32:
        m = [randn(n, seed + 7 * i + 1, 3e-4, off) for i, n in enumerate(sizes)]
        v = [randn(n, seed + 7 * i + 2, 1e-3, off).square() for i, n in enumerate(sizes)]
        if off:
            v = [torch.cat([t.new_zeros(off), t])[off:] for t in v]
        return theta, grads, {"m": m, "v": v}
    codes = lambda i, n, k: torch.randint(0, 256, (n + off,), generator=gen(seed + 7 * i + k), device=DEV,
                                          dtype=torch.uint8)[off:]
    fix = lambda c: torch.where((c & 0x7F) == 0x7F, c - 1, c)       # e4m3's NaN is never written
    scales = lambda i, n, k: torch.randint(100, 110, (-(-n // 128) + off,), generator=gen(seed + 7 * i + k), device=DEV,
                                           dtype=torch.uint8)[off:]
    m = [fix(codes(i, n, 1)) for i, n in enumerate(sizes)]
    if off:
        m = [torch.cat([t.new_zeros(off), t])[off:] for t in m]
    return theta, grads, {"m": m, "v": [codes(i, n, 2) for i, n in enumerate(sizes)],
                          "m_scales": [scales(i, n, 3) for i, n in enumerate(sizes)],
                          "v_scales": [scales(i, n, 4) for i, n in enumerate(sizes)]}


def restored(state, i):
    """(m, root) of tensor i's 8-bit moments by their formats' definitions."""
    s = torch.exp2(state["m_scales"][i].double() - 127).repeat_interleave(128)[:state["m"][i].numel()]
    m = state["m"][i].contiguous().clone().view(torch.float8_e4m3fn).double() * s
    c = state["v"][i].double()
    e = torch.floor(c / 16)
    r = torch.where(e == 0, c / 16 * 2.0 ** -14, (1 + (c - 16 * e) / 16) * torch.exp2(e - 15))
    r = r * torch.exp2(state["v_scales"][i].double() - 127).repeat_interleave(128)[:c.numel()]
    return m.float().cpu().numpy(), r.float().cpu().numpy()


SETS = [[1], [3, 128, 127], [129, 4095], [4096], [4097, 0, 5], [20000, 1, 1, 8192], [0]]


@pytest.mark.parametrize("sizes", SETS, ids=str)
@pytest.mark.parametrize("kind,k", [("f32", 1), ("bf16", 1), ("f16", 3), ("bf16", 4), ("f32", 17)])
@pytest.mark.parametrize("off", [0, 1])
def test_32_bit_moments(rp, sizes, kind, k, off):
    theta, grads, st = problem(sizes, k, kind, 11 * len(sizes) + k, off)
    decay = [0.1 if i % 2 else 0.0 for i in range(len(sizes))]
    order = [(5 * c + 2) % k for c in range(k)] if k != 5 else list(range(k))
    scale = torch.tensor([0.37], device=DEV) if k == 3 else None
    was = [(host(t), [host(grads[c][i]) for c in order], host(st["m"][i]), host(st["v"][i]))
           for i, t in enumerate(theta)]
    rp.adamw(theta, grads if k > 1 else grads[0], **st, step=7, lr=3e-3, weight_decay=decay, order=order,
             grad_scale=scale, **HYPER)
    sc = ref.scalars(7, 3e-3, HYPER["betas"])
    for i, (t, g, m, v) in enumerate(was):
        want = ref.step(t, g, m, v, sc, decay[i], HYPER["betas"], HYPER["eps"], None if scale is None else 0.37)
        assert same(host(theta[i]), want[0]) and same(host(st["m"][i]), want[1]) and same(host(st["v"][i]), want[2])
        if scale is None:
            for got, (val, bound) in zip((theta[i], st["m"][i], st["v"][i]),
                                         ref.step64(*(a.astype(np.float64) if isinstance(a, np.ndarray) else a
                                                      for a in (t, g, m, v)), 7, 3e-3, decay[i], **HYPER)):
                assert (np.abs(host(got) - val) <= bound).all()


@pytest.mark.parametrize("sizes", SETS, ids=str)
@pytest.mark.parametrize("kind,k", [("f32", 1), ("bf16", 4), ("f16", 3)])
@pytest.mark.parametrize("off", [0, 1])
def test_8_bit_moments(rp, sizes, kind, k, off):
    theta, grads, st = problem(sizes, k, kind, 13 * len(sizes) + k, off, bits=8)
    was = [(host(t), [host(g[i]) for g in grads], *restored(st, i)) for i, t in enumerate(theta)]
    for i, n in enumerate(sizes):           # the library's own reading of the codes
        m, v = rp.adamw_moments(st["m"][i], st["v"][i], st["m_scales"][i], st["v_scales"][i])
        assert same(host(m), was[i][2]) and same(host(v), was[i][3] * was[i][3])
    rp.adamw(theta, grads, **st, step=9, lr=1e-3, weight_decay=0.1, seed=5, **HYPER)
    sc = ref.scalars(9, 1e-3, HYPER["betas"], 5)
    for i, (t, g, m, r) in enumerate(was):
        want = ref.step(t, g, m, r * r, sc, 0.1, HYPER["betas"], HYPER["eps"])
        assert same(host(theta[i]), want[0])
        dm, dr = ref.dither(sizes[i], sc[3], i)
        for x, root, d, name in ((want[1], False, dm, "m"), (want[3], True, dr, "v")):
            values, scale = ref.coded(x, root, d)
            got = restored(st, i)[int(root)]
            assert np.array_equal(host(st[name + "_scales"][i]).astype(np.uint8), scale)
            assert same(got, values), name


def test_many_tensors_take_several_launches(rp):
    """1000 tensors do not fit one launch's table: the same results as one at a
    time, and the dither is keyed by the place in the call."""
    sizes = [1 + (37 * i) % 300 for i in range(1000)]
    for bits in (32, 8):
        theta, grads, st = problem(sizes, 1, "f32", 3, bits=bits)
        one = [t.clone() for t in theta]
        st1 = {k: [t.clone() for t in ts] for k, ts in st.items()}
        rp.adamw(theta, grads[0], **st, step=3, lr=1e-2, **HYPER)
        for i in range(1000):
            if bits == 32:
                rp.adamw(one[i], grads[0][i], **{k: ts[i] for k, ts in st1.items()}, step=3, lr=1e-2, **HYPER)
                assert torch.equal(one[i], theta[i])
                assert all(torch.equal(st1[k][i], st[k][i]) for k in st)
            elif i % 100 == 99:
                m, r = restored(st1, i)
                want = ref.step(host(one[i]), [host(grads[0][i])], m, r * r, ref.scalars(3, 1e-2, HYPER["betas"]), 0.0,
                                HYPER["betas"], HYPER["eps"])
                dm, dr = ref.dither(sizes[i], ref.scalars(3, 1e-2, HYPER["betas"])[3], i)
                got = restored(st, i)
                assert same(got[0], ref.coded(want[1], False, dm)[0]) and same(got[1], ref.coded(want[3], True, dr)[0])


def test_zero_state_and_extreme_values(rp):
    """Zeroed memory is a valid start; infinities, NaN, subnormals and huge values
    spoil no group but their own."""
    n = 128 * 6 + 17
    g = randn(n, 1)
    g[0], g[130], g[300], g[301], g[520], g[521] = np.inf, np.nan, 1e30, 1e-30, 1e-42, 0.0
    g[384:512] = 0.0
    for bits in (32, 8):
        theta = randn(n, 2)
        st = rp.adamw_state([theta], bits)
        was = host(theta)
        rp.adamw([theta], [g], **st, step=1, lr=1e-3, **HYPER)
        want = ref.step(was, [host(g)], np.zeros(n, F32), np.zeros(n, F32), ref.scalars(1, 1e-3, HYPER["betas"]), 0.0,
                        HYPER["betas"], HYPER["eps"])
        assert same(host(theta), want[0])
        if bits == 8:
            sc = ref.scalars(1, 1e-3, HYPER["betas"])
            dm, dr = ref.dither(n, sc[3], 0)
            m, v = rp.adamw_moments(st["m"][0], st["v"][0], st["m_scales"][0], st["v_scales"][0])
            wm, wr = ref.coded(want[1], False, dm)[0], ref.coded(want[3], True, dr)[0]
            with np.errstate(over="ignore"):
                assert same(host(m), wm) and same(host(v), wr * wr)
            assert np.isnan(host(m)[:256]).all() and np.isfinite(host(m)[256:]).all()
            assert (host(m)[384:512] == 0).all()
            rp.adamw([theta], [torch.zeros_like(g)], **st, step=2, lr=1e-3, **HYPER)     # and it stays so
            # (1e30 squared is past binary32: its group's roots hold an infinity, and the
            # next step's root is NaN there)
            assert np.isnan(host(theta)[:384]).all() and np.isfinite(host(theta)[384:]).all()


def test_rounding_is_right_on_average(rp):
    """N codes of one value off the grid: each is one of its two neighbours, and
    their mean is within five standard errors of it (a dither's grain is 2^-16)."""
    n = 1 << 16
    g = torch.full((n,), 0.8125 * 1.03, device=DEV)
    g[::128] = 1.75                                     # sets every group's scale
    theta = torch.zeros(n, device=DEV)
    st = rp.adamw_state([theta], 8)
    rp.adamw([theta], [g], **st, step=1, lr=0.0, betas=(0.0, 0.0), eps=1e-8, seed=11)
    m, v = (host(t) for t in rp.adamw_moments(st["m"][0], st["v"][0], st["m_scales"][0], st["v_scales"][0]))
    x = float(F32(0.8125 * 1.03))
    for got, width in ((m, 2.0 ** -4), (np.sqrt(v), 2.0 ** -5)):
        got = np.delete(got, np.arange(0, n, 128)).astype(np.float64)
        low = np.floor(x / width) * width
        assert set(np.round(got / width)) == {round(low / width), round(low / width) + 1}
        p = (x - low) / width
        assert abs(got.mean() - x) <= 5 * width * np.sqrt(p * (1 - p) / len(got)) + width * 2.0 ** -16


def test_nothing_behind_a_tensor_is_written(rp):
    for bits in (32, 8):
        buf = torch.full((3 * 1024,), 7.0, device=DEV)
        theta = buf[512:512 + 333]
        kept = {k: torch.full((2048,), 9, device=DEV, dtype=torch.float32 if bits == 32 else torch.uint8) for k in
                ("m", "v", "m_scales", "v_scales")}
        st = {"m": [kept["m"][100:433]], "v": [kept["v"][100:433]]}
        if bits == 8:
            st.update(m_scales=[kept["m_scales"][3:6]], v_scales=[kept["v_scales"][3:6]])
        rp.adamw([theta], [torch.ones(333, device=DEV)], **st, step=1, lr=1e-3)
        assert (buf[:512] == 7).all() and (buf[845:] == 7).all()
        for k in ("m", "v"):
            assert (kept[k][:100] == 9).all() and (kept[k][433:] == 9).all()
        for k in ("m_scales", "v_scales"):
            assert (kept[k][:3] == 9).all() and (kept[k][6:] == 9).all()


def test_a_replayed_graph_takes_new_scalars_each_step(rp):
    sizes = [1000, 5, 9000]
    for bits in (32, 8):
        theta, grads, st = problem(sizes, 2, "f32", 21, bits=bits)
        eager = [t.clone() for t in theta]
        st2 = {k: [t.clone() for t in ts] for k, ts in st.items()}
        words = rp.adamw_scalars(1, 1e-3, HYPER["betas"]).cuda()
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=other):
            rp.adamw(theta, grads, **st, scalars=words, weight_decay=0.1, **HYPER)
        for step in (4, 5, 6):
            words.copy_(rp.adamw_scalars(step, 1e-3 * step, HYPER["betas"]))
            graph.replay()
            rp.adamw(eager, grads, **st2, step=step, lr=1e-3 * step, weight_decay=0.1, **HYPER)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(theta, eager))
        assert all(torch.equal(a, b) for k in st for a, b in zip(st[k], st2[k]))


def test_another_stream(rp):
    theta, grads, st = problem([50000, 3], 1, "f32", 31)
    a = [t.clone() for t in theta]
    sa = {k: [t.clone() for t in ts] for k, ts in st.items()}
    rp.adamw(theta, grads[0], **st, step=2, lr=1e-3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    rp.adamw(a, grads[0], **sa, step=2, lr=1e-3, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(theta, a))


def test_refusals(rp):
    ok = lambda: problem([300, 20], 1, "f32", 41)
    theta, grads, st = ok()
    g = grads[0]

    def refused(exc, *args, **kw):
        before = [t.clone() for t in theta]
        with pytest.raises(exc):
            rp.adamw(*args, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(before, theta))

    one = dict(step=1, lr=1e-3)
    refused(ValueError, [theta[0].double()] + theta[1:], g, **st, **one)
    refused(ValueError, theta, g[:1], **st, **one)
    refused(ValueError, theta, [g[0][:-1], g[1]], **st, **one)
    refused(ValueError, theta, g, m=st["m"][::-1], v=st["v"], **one)
    refused(ValueError, theta, [g[0].cpu(), g[1]], **st, **one)
    refused(ValueError, theta, g, m=st["m"], v=st["v"], m_scales=st["m"], **one)
    refused(ValueError, theta, g, **st, weight_decay=[0.1], **one)
    refused(ValueError, theta, g, **st, lr=1e-3)
    refused(ValueError, theta, g, **st, order=[0, 1], **one)
    refused(rp.RepopsError, theta, [g, g], **st, order=[0, 0], **one)
    refused(rp.RepopsError, theta, g, **st, step=0, lr=1e-3)
    refused(rp.RepopsError, theta, g, **st, betas=(1.0, 0.9), **one)
    refused(rp.RepopsError, theta, g, **st, eps=float("nan"), **one)
    # a tensor given twice, tensors that overlap, a gradient that is theta itself
    refused(rp.RepopsError, [theta[0], theta[0]], [g[0], g[0]], m=[st["m"][0], st["v"][0]],
            v=[st["m"][0].clone(), st["m"][0].clone()], **one)
    refused(rp.RepopsError, [theta[0][:200], theta[0][199:299]], [g[0][:200], g[0][:100]],
            m=[st["m"][0][:200], st["m"][0][200:300]], v=[st["v"][0][:200], st["v"][0][200:300]], **one)
    refused(rp.RepopsError, theta, theta, **st, **one)
    rp.adamw([], [], m=[], v=[], **one)                       # no tensors: nothing to do
    rp.adamw(theta, [g, g], **st, **one)                      # one gradient for two contributors is fine
