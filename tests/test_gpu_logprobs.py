"""Token log probabilities on the GPU: bit for bit against the step-by-step
definition, and against binary64 with the roundings counted; widths from one
column to many segments, rows on and off 16-byte boundaries, few rows (a cluster
each) and many, masked and empty rows, infinities and NaN, ties, streams, graphs
and refusals; the gradient against the formula's and against differences."""
import numpy as np
import pytest
import torch

import logprobs_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32 = np.float32
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
WIDTHS = [1, 2, 31, 33, 255, 256, 257, 1000, 1023, 1024, 1025, 2047, 4097, 9001, 40000]


def host(t):
    return t.detach().float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def same(a, b):
    a, b = np.asarray(a, F32), np.asarray(b, F32)
    both = np.isnan(a) & np.isnan(b)
    return a.shape == b.shape and np.array_equal(np.where(both, 0, a).view(np.uint32), np.where(both, 0, b).view(np.uint32))


def logits(rows, cols, kind, seed, pad=0, off=0, sd=3.0):
    """rows x cols at pitch cols + pad, the first `off` values behind the start of memory."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    flat = (torch.randn(max(rows * (cols + pad), 1) + off, generator=g, device=DEV) * sd).to(DT[kind])
    return flat.as_strided((rows, cols), (cols + pad, 1), off)


def some_targets(rows, cols, seed):
    t = torch.randint(0, cols, (rows,), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)
    if rows > 2:
        t[1] = -100
    return t


def check(rp, x, targets, temperature, top):
    """token_logprobs against the definition, every output, bit for bit."""
    got = rp.token_logprobs(x, targets, temperature=temperature, top=top)
    want = ref.forward(host(x), None if targets is None else host(targets), temperature, top)
    for name, w in zip(("logp", "lse", "entropy", "stats"), want):
        assert same(host(getattr(got, name)), w), name
    if top:
        assert same(host(got.top_logp), want[4])
        assert np.array_equal(host(got.top_ids), want[5])
    else:
        assert got.top_logp is None and got.top_ids is None
    return got


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_the_definition(rp, cols, kind):
    for rows, pad, off, T, top in ((1, 0, 0, 1.0, 1), (5, 0, 0, 0.7, 8), (3, 1, 1, 1.3, 32), (4, 5, 3, 1.0, 0),
                                   (2, 8, 0, 2.0, 5), (9, 3, 7, 1.0, 2)):
        x = logits(rows, cols, kind, cols + rows, pad, off)
        if cols > 40:
            x[:, 7:19] = -np.inf                            # impossible tokens
        check(rp, x, some_targets(rows, cols, rows), T, min(top, cols))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_few_rows_share_a_row_between_ctas(rp, kind):
    """1 to 700 rows of one matrix: every cluster size gives a row the same bits."""
    x = logits(700, 20011, kind, 5)
    t = some_targets(700, 20011, 6)
    whole = rp.token_logprobs(x, t, top=7)
    for rows in (1, 2, 40, 80, 160, 320):
        part = rp.token_logprobs(x[:rows], t[:rows], top=7)
        for a, b in zip(part, whole):
            assert torch.equal(a, b[:rows]), rows
    pick = torch.tensor([0, 1, 333, 699])
    want = ref.forward(host(x[pick]), host(t[pick]), 1.0, 7)
    for a, w in zip(whole, want):
        assert same(host(a[pick]), w) if a.is_floating_point() else np.array_equal(host(a[pick]), w)


@pytest.mark.parametrize("cols", [1, 33, 257, 1024, 5001])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1.0, 0.5])
def test_against_binary64(rp, cols, kind, T):
    x = logits(20, cols, kind, 7 * cols)
    if cols > 40:
        x[3:9, 5:30] = -np.inf
    t = some_targets(20, cols, cols)
    if cols > 40:
        t[4] = 6                                            # an impossible target
    got = rp.token_logprobs(x, t, temperature=T)
    f = ref.forward64(host(x), host(t), T)[0]
    for name, (val, bound) in f.items():
        g = host(getattr(got, name)).astype(np.float64)
        assert np.array_equal(np.isinf(g), np.isinf(val)) and np.array_equal(g[np.isinf(g)], val[np.isinf(val)])
        fin = np.isfinite(val)
        assert (np.abs(g[fin] - val[fin]) <= bound[fin]).all(), name
    g = torch.Generator(device=DEV).manual_seed(3)
    dl, de = (torch.randn(20, generator=g, device=DEV) for _ in range(2))
    for a, b in ((dl, None), (None, de), (dl, de)):
        d = rp.token_logprobs_backward(x, t, got.stats, a, b, temperature=T)
        val, bound = ref.backward64(host(x), host(t), None if a is None else host(a), None if b is None else host(b), T)
        # half a step of the storage type, and half its smallest subnormal
        bound = bound + np.abs(val) * EPS[kind] + {"f32": 0, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[kind]
        assert (np.abs(host(d).astype(np.float64) - val) <= bound).all()


@pytest.mark.parametrize("cols", [1, 31, 256, 1025, 9001])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad,off,opad", [(0, 0, 0), (3, 1, 3), (1, 0, 2), (8, 5, 16)])
def test_gradient_definition(rp, cols, kind, pad, off, opad):
    rows, T = 4, 0.8
    x = logits(rows, cols, kind, cols + 1, pad, off)
    if cols > 40:
        x[:, 7:19] = -np.inf
        x[2] = -np.inf                                      # a row with nothing possible
    t = some_targets(rows, cols, 9)
    st = rp.token_logprobs(x, t, temperature=T).stats
    g = torch.Generator(device=DEV).manual_seed(4)
    dl, de = (torch.randn(rows, generator=g, device=DEV) for _ in range(2))
    for a, b in ((dl, None), (None, de), (dl, de)):
        buf = torch.full((rows * (cols + opad) + off,), 7.0, dtype=DT[kind], device=DEV)
        out = buf.as_strided((rows, cols), (cols + opad, 1), off)
        rp.token_logprobs_backward(x, t, st, a, b, temperature=T, out=out)
        want = ref.backward(host(x), host(t), host(st), None if a is None else host(a), None if b is None else host(b), T)
        want = host(torch.from_numpy(want).to(DT[kind]))
        assert same(host(out), want)
        left = buf.clone()
        left.as_strided((rows, cols), (cols + opad, 1), off).fill_(7.0)
        assert (left == 7).all()                            # nothing but its rows was written
        y = x.clone(memory_format=torch.preserve_format)
        assert rp.token_logprobs_backward(y, t, st, a, b, temperature=T, out=y) is y and same(host(y), want)


def test_gradient_is_the_difference_quotient(rp):
    """logp and entropy of two nearby logits, in the direction of one of them: the
    library's own forward in binary32 resolves 2^-22 of values about 8, so a step of
    2^-6 leaves 2^-15 and the curvature (third derivative below 1) 2^-13 / 6."""
    rows, cols, step = 6, 300, 2.0 ** -6
    x = torch.round(logits(rows, cols, "f32", 12) * 64) / 64        # so that both steps are exact
    t = torch.arange(rows, device=DEV) * 3
    one = torch.ones(rows, device=DEV)
    st = rp.token_logprobs(x, t).stats
    dl, de = (rp.token_logprobs_backward(x, t, st, a, b) for a, b in ((one, None), (None, one)))
    for j in (0, 3, 15, 299):
        d = torch.zeros_like(x)
        d[:, j] = step
        up, dn = rp.token_logprobs(x + d, t), rp.token_logprobs(x - d, t)
        for g, a, b in ((dl, up.logp, dn.logp), (de, up.entropy, dn.entropy)):
            assert ((a - b) / (2 * step) - g[:, j]).abs().max() <= 2.0 ** -13 + 2.0 ** -12


def test_empty_infinite_and_nan_rows(rp):
    for kind in ("f32", "f16", "bf16"):
        for cols in (5, 1030, 3000):
            x = logits(8, cols, kind, 3)
            x[0] = -np.inf
            x[1], x[1, 4] = -np.inf, 2.0                    # one possibility: certain
            x[2, 3] = np.nan
            x[3, 2] = np.inf
            x[4, cols - 1], x[4, 0] = np.nan, np.inf
            x[5] = 1.5                                      # all alike
            x[6, 1::2], x[6, 0::2] = 0.0, -0.0
            t = torch.tensor([1, 4, 0, 1, 2, cols - 1, 3, cols], device=DEV)
            got = check(rp, x, t, 1.0, min(5, cols))
            assert host(got.logp)[0] == -np.inf and host(got.lse)[0] == -np.inf and host(got.entropy)[0] == 0
            assert host(got.logp)[1] == 0 and host(got.entropy)[1] == 0
            assert np.isnan(host(got.logp)[[2, 3, 4, 7]]).all() and np.isnan(host(got.entropy)[2:5]).all()
            assert host(got.top_ids)[5].tolist() == [0, 1, 2, 3, 4] and host(got.top_ids)[6].tolist() == [0, 1, 2, 3, 4]
            w = torch.ones(8, device=DEV)
            d = host(rp.token_logprobs_backward(x, t, got.stats, w, w))
            assert (d[0] == 0).all() and (d[1] == 0).all() and np.isnan(d[[2, 3, 4, 7]]).all()
            assert np.isfinite(d[[5, 6]]).all()


def test_ties_across_segments(rp):
    """Alternatives are the lowest columns among equals, wherever they lie."""
    for kind in ("f32", "bf16"):
        x = torch.zeros(3, 50000, dtype=DT[kind], device=DEV)
        x[0, [49999, 1024, 30000, 5, 1023]] = 3.0
        x[1, 1024 * 7:1024 * 8] = 2.0
        x[1, [40000, 20000, 1]] = 4.0
        got = check(rp, x, None, 1.0, 32)
        assert host(got.top_ids)[0, :6].tolist() == [5, 1023, 1024, 30000, 49999, 0]
        assert host(got.top_ids)[1, :5].tolist() == [1, 20000, 40000, 7168, 7169]
        assert host(got.top_ids)[2].tolist() == list(range(32))


def test_no_rows_other_streams_and_graphs(rp):
    r = rp.token_logprobs(torch.empty(0, 77, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV), top=3)
    assert r.logp.shape == (0,) and r.top_ids.shape == (0, 3)
    x, t = logits(30, 7001, "bf16", 8), some_targets(30, 7001, 9)
    w = torch.randn(30, device=DEV)
    a = rp.token_logprobs(x, t, top=4)
    da = rp.token_logprobs_backward(x, t, a.stats, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = rp.token_logprobs(x, t, top=4)
        db = rp.token_logprobs_backward(x, t, b.stats, w)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and torch.equal(da, db)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = rp.token_logprobs(x, t, top=4)
        dc = rp.token_logprobs_backward(x, t, c.stats, w)
    for seed in (20, 21):
        x.copy_(logits(30, 7001, "bf16", seed))
        graph.replay()
        d = rp.token_logprobs(x, t, top=4)
        assert all(torch.equal(p, q) for p, q in zip(c, d))
        assert torch.equal(dc, rp.token_logprobs_backward(x, t, d.stats, w))


def test_refusals(rp):
    x, t = logits(4, 100, "f32", 1), some_targets(4, 100, 1)
    st = rp.token_logprobs(x, t).stats
    w = torch.ones(4, device=DEV)
    for bad in (dict(top=33), dict(top=-1), dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan"))):
        with pytest.raises(rp.RepopsError):
            rp.token_logprobs(x, t, **bad)
    with pytest.raises(rp.RepopsError):
        rp.token_logprobs(x[:, :5], t, top=6)
    with pytest.raises(rp.RepopsError):
        rp.token_logprobs(x[:, :0], t)
    for args in ((x.t(), t), (x, t.int()), (x, t[:3]), (x[0], t), (x[:1].expand(4, 100), t), (x, t.cpu()), (x.cpu(), t)):
        with pytest.raises(ValueError):
            rp.token_logprobs(*args)
    with pytest.raises(TypeError):
        rp.token_logprobs(x.double(), t)
    with pytest.raises(rp.RepopsError):
        rp.token_logprobs_backward(x, t, st)                 # no gradient given
    with pytest.raises(rp.RepopsError):
        rp.token_logprobs_backward(x, None, st, w)           # whose log probabilities?
    with pytest.raises(rp.RepopsError):
        rp.token_logprobs_backward(x[:3], t[:3], st[:3], w[:3], out=x[1:])    # another row's memory
    for bad in ((x, t, st[:3], w), (x, t, st, w[:3]), (x, t, st, w.double()), (x, t, st.t().contiguous().t(), w)):
        with pytest.raises(ValueError):
            rp.token_logprobs_backward(*bad)
    with pytest.raises(ValueError):
        rp.token_logprobs_backward(x, t, st, w, out=torch.empty(4, 100, dtype=torch.float16, device=DEV))
