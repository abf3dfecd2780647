"""Plain NumPy statements of the 8-bit row format and of the block edge, for
the tests: the format bit for bit in binary32, the rest in binary64."""
import numpy as np

F32 = np.float32
FLOOR = F32(2.0 ** -100)


def quantize(x, group):
    """(q, scale) of the rows of a float32 array, step by step in binary32."""
    rows, cols = x.shape
    width = group or max(cols, 1)
    n = -(-cols // width) if group else 1
    q = np.zeros((rows, cols), np.int8)
    scale = np.zeros((rows, n), F32)
    with np.errstate(all="ignore"):
        for r in range(rows):
            for j in range(n):
                part = x[r, j * width:(j + 1) * width].astype(F32)
                if not np.isfinite(part).all():
                    scale[r, j] = np.nan
                    continue
                a = max(np.abs(part).max(initial=F32(0)), FLOOR)
                scale[r, j] = F32(a) / F32(127)
                q[r, j * width:(j + 1) * width] = np.rint(part * (F32(127) / F32(a))).astype(np.int8)
    return q, scale


def dequantize(q, scale, group):
    cols = q.shape[1]
    s = np.repeat(scale, group, axis=1)[:, :cols] if group else np.broadcast_to(scale, q.shape)
    return q.astype(F32) * s


def norm64(v, gain, eps):
    inv = 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    return v * inv, inv, v * inv * gain


def norm_grad64(v, gain, d, eps):
    """(dv, terms of dgain, a magnitude bound of dv): every sum with its terms'
    absolute values."""
    vh, inv, _ = norm64(v, gain, eps)
    g = d * gain
    dv = inv * (g - vh * (g * vh).mean(1, keepdims=True))
    mag = inv * (np.abs(g) + np.abs(vh) * np.abs(g * vh).mean(1, keepdims=True))
    return dv, d * vh, mag


def edge64(x, f, post, gate, alpha, pre, eps):
    """(y, h): the forward in binary64; gate already one row per row."""
    p = f if post is None else norm64(f, post, eps)[2]
    t = p if gate is None else p * gate
    y = x + alpha * t
    return y, None if pre is None else norm64(y, pre, eps)[2]


def edge_backward64(dy, dh, y, f, post, gate, alpha, pre, eps, gates):
    """The gradients in binary64 and, beside each, the magnitude its rounding
    errors are relative to: {name: (value, magnitude)}."""
    out = {}
    if pre is None:
        dx, mdx = dy, np.abs(dy)
    else:
        dx, terms, mdx = norm_grad64(y, pre, dh, eps)
        out["dpre"] = (terms.sum(0), np.abs(terms).sum(0))
        if dy is not None:
            dx, mdx = dx + dy, mdx + np.abs(dy)
    out["dx"] = (dx, mdx)
    dt, mdt = alpha * dx, abs(alpha) * mdx
    dp = dt if gate is None else dt * gate
    mdp = mdt if gate is None else mdt * np.abs(gate)
    if post is None:
        out["df"] = (dp, mdp)
        p = f
    else:
        df, terms, _ = norm_grad64(f, post, dp, eps)
        fh, inv, p = norm64(f, post, eps)
        mg = mdp * np.abs(post)
        out["df"] = (df, inv * (mg + np.abs(fh) * (mg * np.abs(fh)).mean(1, keepdims=True)))
        out["dpost"] = (terms.sum(0), (mdp * np.abs(fh)).sum(0))
    if gate is not None:
        split = lambda a: a.reshape(gates, -1, a.shape[1]).sum(1)
        out["dgate"] = (split(dt * p), split(mdt * np.abs(p)))
    return out
