"""Plain NumPy statements of head norms with the rotation, for the tests: the
binary32 definition step by step (the library's bits), and binary64."""
import numpy as np

F32 = np.float32
U = 2.0 ** -24


def tree(v):
    """The 32-ary tree over the last axis."""
    while v.shape[-1] > 1:
        n = v.shape[-1]
        out = []
        for s in range(0, n, 32):
            acc = v[..., s]
            for i in range(s + 1, min(s + 32, n)):
                acc = acc + v[..., i]
            out.append(acc)
        v = np.stack(out, -1)
    return v[..., 0]


def pairs_of(pairs, layout):
    i = np.arange(pairs)
    return (2 * i, 2 * i + 1) if layout == "adjacent" else (i, i + pairs)


def table_rows(cos, sin, pos):
    """cos and sin of each row's position: NaN past the table, 1 and 0 for rows left alone."""
    out = []
    for t, none in ((cos, 1), (sin, 0)):
        v = t[np.clip(pos, 0, len(t) - 1)].copy()
        v[pos >= len(t)] = np.nan
        v[pos < 0] = none
        out.append(v[:, None, :])
    return out


def rotate(x, cos, sin, pos, layout, back):
    """x: rows x heads x dim of any float type, the table's values converted to it."""
    a, b = pairs_of(cos.shape[1], layout)
    c, s = (t.astype(x.dtype) for t in table_rows(cos, sin, pos))
    y = x.copy()
    u, v = x[..., a], x[..., b]
    y[..., a] = u * c + v * s if back else u * c - v * s
    y[..., b] = v * c - u * s if back else u * s + v * c
    return y


def inv32(x, eps):
    ms = tree(x * x) / F32(x.shape[-1])
    return (F32(1) / np.sqrt(ms + F32(eps)))[..., None]


def forward(x, gains, eps, cos, sin, pos, layout, back=False):
    """x: rows x heads x dim binary32; gains: heads x dim or None.  Before narrowing."""
    with np.errstate(all="ignore"):
        v = x if gains is None else (x * inv32(x, eps)) * gains
        return v if cos is None else rotate(v, cos, sin, pos, layout, back)


def backward(dy, x, gains, eps, cos, sin, pos, layout):
    """(dx, terms): rows x heads x dim binary32; terms of rows left alone are +0."""
    with np.errstate(all="ignore"):
        g = dy if cos is None else rotate(dy, cos, sin, pos, layout, True)
        inv = inv32(x, eps)
        xh = x * inv
        gy = g * gains
        c = (tree(gy * xh) / F32(x.shape[-1]))[..., None]
        terms = g * xh
        terms[pos < 0] = 0
        return inv * (gy - xh * c), terms


def colsum(terms):
    """The column sums of rows x heads x dim terms over (row, head) in order."""
    t = terms.reshape(-1, terms.shape[-1])
    return tree(np.ascontiguousarray(t.T)) if len(t) else np.zeros(terms.shape[-1], F32)


def forward64(x, gains, eps, cos, sin, pos, layout):
    """(value, bound): a value's error is at most seven roundings (the sum's tree as
    three, the norm's four) on its product and three on the rotation's terms."""
    x = x.astype(np.float64)
    v = x if gains is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gains.astype(np.float64)
    n = 0 if gains is None else x.shape[-1] / 2 + 8        # the sum's worst case: half a step an addition
    if cos is None:
        return v, np.abs(v) * n * U + 1e-37
    y = rotate(v, cos.astype(np.float64), sin.astype(np.float64), pos, layout, False)
    m = np.abs(v) * (n + 3) * U
    a, b = pairs_of(cos.shape[1], layout)
    bound = m.copy()
    bound[..., a] = m[..., a] + m[..., b]
    bound[..., b] = m[..., a] + m[..., b]
    return y, bound + 1e-37


def backward64(dy, x, gains, eps, cos, sin, pos, layout):
    """(dx, bound), (terms, bound) in binary64."""
    dy, x, gains = (t.astype(np.float64) for t in (dy, x, gains))
    g, mg = dy, np.abs(dy)
    if cos is not None:
        g = rotate(dy, cos.astype(np.float64), sin.astype(np.float64), pos, layout, True)
        a, b = pairs_of(cos.shape[1], layout)
        mg = mg.copy()
        mg[..., a] = mg[..., b] = np.abs(dy[..., a]) + np.abs(dy[..., b])
    d = x.shape[-1]
    inv = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * inv
    gy, mgy = g * gains, mg * np.abs(gains)
    c = (gy * xh).mean(-1, keepdims=True)
    mc = (mgy * np.abs(xh)).mean(-1, keepdims=True)
    n = 2 * d + 24                       # two sums of d terms, and each value's steps
    dx = inv * (gy - xh * c)
    terms = g * xh
    terms[pos < 0] = 0
    return (dx, inv * (mgy + np.abs(xh) * mc) * n * U + 1e-37), (terms, mg * np.abs(xh) * (d / 2 + 12) * U)
