"""The edge between two blocks on the GPU: forward and backward against the
composition of the library's separate operators (bit for bit) and against the
formulas in binary64, over widths from one value to several tree levels, gates
a vector, a sequence and a token, pitches, in-place calls and missing operands."""
import numpy as np
import pytest
import torch

from verifiable_repops_gemm_gb300 import inputs

import rows8_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 1e-5
U = 2.0 ** -24
SIZES = [(1, 1), (1, 2048), (3, 5), (6, 33), (33, 100), (96, 1023), (64, 1024), (66, 2048), (3, 4100), (6, 8192),
         (3, 8193), (33, 9001)]


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int32), b.contiguous().view(torch.int32))


def normal(shape, sd, seed, pad=0):
    rows, cols = shape
    return inputs.normal((rows, cols + pad), sd, seed, DEV)[:, :cols]


def operands(rows, cols, gates, post, seed, pad=0):
    gain = lambda k: 1.0 + 0.1 * inputs.normal((cols,), 1.0, seed + k, DEV)
    return {"x": normal((rows, cols), 1.0, seed, pad), "f": normal((rows, cols), 3.0, seed + 1, pad),
            "pre": gain(2), "post": gain(3) if post else None,
            "gate": 0.5 + 0.2 * normal((gates, cols), 1.0, seed + 4, pad) if gates else None}


def spread(gate, rows):
    return None if gate is None else gate.repeat_interleave(rows // gate.shape[0], 0)


def composed(rp, o, alpha):
    """The separate operators: rmsnorm_rows and element-wise steps."""
    rows, cols = o["x"].shape
    p = o["f"] if o["post"] is None else rp.rmsnorm_rows(o["f"], o["post"], EPS)
    t = p if o["gate"] is None else p * spread(o["gate"], rows)
    y = o["x"] + t * alpha
    return p, y.contiguous(), rp.rmsnorm_rows(y.contiguous(), o["pre"], EPS)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("post,gates,alpha", [(True, 1, 0.5), (False, 0, 1.0), (True, 3, -0.3), (False, -1, 1.0)])
def test_forward_equals_the_separate_operators(rp, rows, cols, post, gates, alpha):
    gates = rows if gates < 0 else gates if rows % max(gates, 1) == 0 else 1
    for pad in (0, 3, 4):
        o = operands(rows, cols, gates, post, rows + cols, pad)
        _, wy, wh = composed(rp, o, alpha)
        y, h = rp.rmsnorm_residual(o["x"], o["f"], o["pre"], EPS, post_gain=o["post"], gate=o["gate"], alpha=alpha)
        assert same(y, wy) and same(h, wh)
        y, h = rp.rmsnorm_residual(o["x"], o["f"], None, EPS, post_gain=o["post"], gate=o["gate"], alpha=alpha)
        assert h is None and same(y, wy)
        x2, f2 = o["x"].clone(), o["f"].clone()
        rp.rmsnorm_residual(x2, f2, o["pre"], EPS, post_gain=o["post"], gate=o["gate"], alpha=alpha, y=x2, h=f2)
        assert same(x2, wy) and same(f2, wh)                       # both results in place


def composed_backward(rp, o, dy, dh, y, alpha, gates):
    rows, cols = o["f"].shape
    if dh is None:
        dx, dpre = dy, None
    else:
        dx, t = rp.rmsnorm_backward(y, o["pre"], EPS, dh, res=dy)
        dpre = rp.colsum(t)
    dt = dx * alpha
    dp = dt if o["gate"] is None else dt * spread(o["gate"], rows)
    dp = dp.contiguous()
    p, df, dpost, dgate = o["f"], dp, None, None
    if o["post"] is not None:
        df, t = rp.rmsnorm_backward(o["f"], o["post"], EPS, dp)
        dpost = rp.colsum(t)
        p = rp.rmsnorm_rows(o["f"], o["post"], EPS)
    if o["gate"] is not None:
        terms = (dt * p).contiguous()
        per = rows // gates
        dgate = torch.stack([rp.colsum(terms[g * per:(g + 1) * per]) for g in range(gates)])
    return dx, df, dpre, dpost, dgate


@pytest.mark.parametrize("rows,cols", SIZES + [(33000, 8), (32 * 5, 64)])
@pytest.mark.parametrize("post,gates,alpha", [(True, 1, 0.5), (False, 0, 1.0), (True, 3, -0.3), (True, 5, 0.5),
                                              (False, 2, 0.25), (True, -1, 1.0)])
def test_backward_equals_the_separate_operators(rp, rows, cols, post, gates, alpha):
    gates = min(rows, 100) if gates < 0 else gates
    while gates > 1 and rows % gates:
        gates -= 1
    for pad in (0, 3):
        o = operands(rows, cols, gates, post, rows + cols, pad)
        _, y, _ = composed(rp, o, alpha)
        dy, dh = normal((rows, cols), 1.0, 7, pad), normal((rows, cols), 1.0, 8, pad)
        for d, e in ((dy, dh), (None, dh), (dy, None)):
            want = composed_backward(rp, o, d, e, y, alpha, gates)
            got = rp.rmsnorm_residual_backward(d, e, y if e is not None else None, o["f"],
                                               o["pre"] if e is not None else None, EPS, post_gain=o["post"],
                                               gate=o["gate"], alpha=alpha)
            for name, g, w in zip(("dx", "df", "dpre", "dpost", "dgate"), got, want):
                assert (g is None) == (w is None), name
                assert g is None or same(g, w), (name, pad, d is None, e is None)
        d2 = dy.clone()
        got = rp.rmsnorm_residual_backward(d2, dh, y, o["f"], o["pre"], EPS, post_gain=o["post"], gate=o["gate"],
                                           alpha=alpha, dx=d2)                       # in place over dy
        want = composed_backward(rp, o, dy, dh, y, alpha, gates)
        assert got[0] is d2 and all(g is None or same(g, w) for g, w in zip(got, want))


def test_many_rows_of_one_gate(rp):
    """More than 1024 runs of a gate's rows, on two gates: the further level."""
    rows, cols = 2 * 32800, 12
    o = operands(rows, cols, 2, True, 77)
    dy, dh = normal((rows, cols), 1.0, 78), normal((rows, cols), 1.0, 79)
    _, y, _ = composed(rp, o, 0.5)
    got = rp.rmsnorm_residual_backward(dy, dh, y, o["f"], o["pre"], EPS, post_gain=o["post"], gate=o["gate"], alpha=0.5)
    want = composed_backward(rp, o, dy, dh, y, 0.5, 2)
    assert all(same(g, w) for g, w in zip(got, want))


# Rounding errors, in half-steps U relative to the terms' magnitudes (the
# reference gives each): a row's tree folds at most 32 + 32 + 8 sums for these
# widths, so 1/rms is off by (72 + 2) / 2 + 4 < 42 and xhat by 43; the mean of
# gy * xhat by 1 + 43 + 1 + 72 + 1 = 118; a norm's gradient by 118 + 43 + 2 + 42
# = 205; dp adds 3, the second norm's gradient at most 208 + 205 again; a column
# sum adds 73.  512 covers each of them.
@pytest.mark.parametrize("rows,cols,gates", [(33, 100, 1), (64, 2048, 2), (5, 4099, 5)])
def test_against_binary64(rp, rows, cols, gates):
    o = operands(rows, cols, gates, True, 90 + cols)
    alpha = 0.37
    y, h = rp.rmsnorm_residual(o["x"], o["f"], o["pre"], EPS, post_gain=o["post"], gate=o["gate"], alpha=alpha)
    n = {k: v.double().cpu().numpy() for k, v in o.items()}
    a32 = float(np.float32(alpha))
    gate = np.repeat(n["gate"], rows // gates, axis=0)
    e32 = float(np.float32(EPS))
    wy, wh = ref.edge64(n["x"], n["f"], n["post"], gate, a32, n["pre"], e32)
    mag = np.abs(n["x"]) + np.abs(wy - n["x"])
    assert (np.abs(y.cpu().numpy() - wy) <= 64 * U * mag).all()
    ynum = y.double().cpu().numpy()
    assert (np.abs(h.cpu().numpy() - ref.norm64(ynum, n["pre"], e32)[2]) <= 64 * U * np.abs(wh) + 1e-30).all()
    dy, dh = normal((rows, cols), 1.0, 91), normal((rows, cols), 1.0, 92)
    got = dict(zip(("dx", "df", "dpre", "dpost", "dgate"), rp.rmsnorm_residual_backward(
        dy, dh, y, o["f"], o["pre"], EPS, post_gain=o["post"], gate=o["gate"], alpha=alpha)))
    want = ref.edge_backward64(dy.double().cpu().numpy(), dh.double().cpu().numpy(), ynum, n["f"], n["post"], gate, a32,
                               n["pre"], e32, gates)
    for name, (w, m) in want.items():
        assert (np.abs(got[name].cpu().numpy() - w) <= 512 * U * m).all(), name


def test_nan_stays_in_its_row(rp):
    o = operands(9, 300, 1, True, 99)
    o["f"][4, 17] = float("nan")
    y, h = rp.rmsnorm_residual(o["x"], o["f"], o["pre"], EPS, post_gain=o["post"], gate=o["gate"])
    bad = torch.isnan(y).any(1) | torch.isnan(h).any(1)
    assert bad.tolist() == [i == 4 for i in range(9)]


def test_no_rows(rp):
    e = torch.empty(0, 64, device=DEV)
    g = torch.ones(64, device=DEV)
    y, h = rp.rmsnorm_residual(e, e.clone(), g, EPS, post_gain=g, gate=g)
    assert y.shape == h.shape == (0, 64)
    out = rp.rmsnorm_residual_backward(e, e, e, e, g, EPS, post_gain=g, gate=g)
    assert all((t == 0).all() for t in out[2:])


def test_captured_graphs_share_nothing(rp):
    o = operands(130, 2048, 2, True, 120)
    dy, dh = normal((130, 2048), 1.0, 121), normal((130, 2048), 1.0, 122)
    kw = dict(post_gain=o["post"], gate=o["gate"], alpha=0.5)
    y, _ = rp.rmsnorm_residual(o["x"], o["f"], o["pre"], EPS, **kw)
    want = rp.rmsnorm_residual_backward(dy, dh, y, o["f"], o["pre"], EPS, **kw)
    graphs = []
    for _ in range(2):
        outs = [torch.zeros_like(t) for t in want]
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            rp.rmsnorm_residual_backward(dy, dh, y, o["f"], o["pre"], EPS, **kw, dx=outs[0], df=outs[1], dpre=outs[2],
                                         dpost=outs[3], dgate=outs[4])
        graphs.append((gr, outs))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for st, (gr, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        assert all(same(a, b) for a, b in zip(outs, want))


def test_rows_that_share_memory_are_refused(rp):
    o = operands(6, 40, 1, True, 130)
    one = o["x"][:1]
    for bad in (dict(x=one.expand(6, 40)), dict(f=one.expand(6, 40)), dict(y=one.expand(6, 40))):
        kw = dict(x=o["x"], f=o["f"], pre_gain=o["pre"], eps=EPS)
        kw.update(bad)
        with pytest.raises(ValueError):
            rp.rmsnorm_residual(**kw)
    with pytest.raises(ValueError):
        rp.rmsnorm_residual(o["x"], o["f"], o["pre"], EPS, gate=o["gate"].expand(3, 40))
    A = torch.ones(4, 64, dtype=torch.int8, device=DEV)
    s = torch.ones(4, device=DEV)
    with pytest.raises(ValueError):
        rp.gemm_i8(A[:1].expand(4, 64), A.t(), s, s)
    with pytest.raises(ValueError):
        rp.gemm_i8(A, A.t(), s, s, out=torch.empty(1, 4, device=DEV).expand(4, 4))
    with pytest.raises(ValueError):
        rp.quantize_rows(one.expand(6, 40))
    with pytest.raises(ValueError):
        rp.dequantize_rows(A, s.view(4, 1), out=torch.empty(1, 64, device=DEV).expand(4, 64))
