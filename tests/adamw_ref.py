"""Plain NumPy statements of the AdamW step and of its 8-bit moments, for the
tests: every step one binary32 rounding, the codes by exact arithmetic on their
values (no bit patterns), and the step in binary64 with its rounding errors."""
import numpy as np

F32 = np.float32
GROUP = 128
M32 = 0xFFFFFFFF


def mix(h):
    h = np.asarray(h, np.uint64) & np.uint64(M32)
    h = ((h ^ (h >> np.uint64(16))) * np.uint64(0x85EBCA6B)) & np.uint64(M32)
    h = ((h ^ (h >> np.uint64(13))) * np.uint64(0xC2B2AE35)) & np.uint64(M32)
    return h ^ (h >> np.uint64(16))


def scalars(step, lr, betas, seed=0):
    b1, b2 = betas
    return (F32(lr), F32(lr / (1 - b1 ** step)), F32(1 / np.sqrt(1 - b2 ** step)),
            int(mix((0x9E3779B9 * step + seed) & M32)))


def dither(n, key, tensor):
    k = int(mix((key + 0x9E3779B9 * (tensor + 1)) & M32))
    h = mix((np.arange(n, dtype=np.uint64) * np.uint64(0x9E3779B1) + np.uint64(k)) & np.uint64(M32))
    return (h & np.uint64(0xFFFF)).astype(np.float64), (h >> np.uint64(16)).astype(np.float64)


def coded(x, root, dith):
    """(values, scale bytes) that the codes of a binary32 array stand for: m's
    format, or a root's.  Groups that are not finite come back as NaN."""
    x = np.asarray(x, F32)
    n = len(x)
    bits, most, low = (4, 1.9375, 112) if root else (3, 448.0, 120)
    groups = -(-n // GROUP)
    scale = np.zeros(groups, np.uint8)
    out = np.empty(n, F32)
    for q in range(groups):
        part = slice(q * GROUP, min(n, (q + 1) * GROUP))
        a = np.abs(x[part]).astype(np.float64)
        if not np.isfinite(a).all():
            scale[q], out[part] = 255, np.nan
            continue
        s = 1
        while a.max() > most * 2.0 ** (s - 127):
            s += 1
        scale[q] = s
        with np.errstate(all="ignore"):
            y = (np.abs(x[part]) * F32(2.0 ** (127 - s))).astype(F32) * F32(2.0 ** -low)
        y = y.astype(np.float64)
        # a code's width: 2^-bits of the value's binade, that of 2^-126 below it
        with np.errstate(divide="ignore"):
            e = np.where(y > 0, np.maximum(np.floor(np.log2(np.where(y > 0, y, 1.0))), -126), -126)
        e = np.where(y >= 2.0 ** (e + 1), e + 1, np.where((y < 2.0 ** e) & (e > -126), e - 1, e))
        width = 2.0 ** (e - bits)
        whole = np.floor(y / width)
        up = (y / width - whole) * 65536 + dith[part] + 0.5 >= 65536
        code = whole + up
        if root:
            code = np.where((y > 0) & (code == 0), 1, code)
        v = code * width * 2.0 ** low * 2.0 ** (int(s) - 127)
        out[part] = (v if root else np.copysign(v, x[part])).astype(F32)
    return out, scale


def step(theta, grads, m, v, sc, decay, betas, eps, grad_scale=None):
    """(theta, m, v, root): grads in the order of the fold."""
    lr, s, b, _ = sc
    b1, c1, b2, c2 = F32(betas[0]), F32(1 - betas[0]), F32(betas[1]), F32(1 - betas[1])
    with np.errstate(all="ignore"):
        g = grads[0].astype(F32)
        for t in grads[1:]:
            g = (g + t.astype(F32)).astype(F32)
        if len(grads) > 1:
            g = (g / F32(len(grads))).astype(F32)
        if grad_scale is not None:
            g = (g * F32(grad_scale)).astype(F32)
        m = m * b1 + g * c1
        v = v * b2 + (g * g) * c2
        r = np.sqrt(v)
        u = m / (r * b + F32(eps))
        keep = F32(1) - F32(decay) * lr
        return theta * keep - u * s, m, v, r


def step64(theta, grads, m, v, n, lr, decay, betas, eps):
    """(value, bound) of theta, m and v in binary64: the bound counts half a step
    (2^-24 of the value) for each rounding on the way, the constants' included."""
    U = 2.0 ** -24
    g = sum(t.astype(np.float64) for t in grads) / len(grads)
    mag = sum(np.abs(t.astype(np.float64)) for t in grads) / len(grads)
    dg = (len(grads) if len(grads) > 1 else 0) * mag * U            # the fold's sums and the divide
    b1, b2 = betas
    m1, m2 = b1 * m, (1 - b1) * g
    mm = m1 + m2
    dm = (2 * np.abs(m1) + 2 * np.abs(m2) + np.abs(m1) + np.abs(m2)) * U + (1 - b1) * dg
    v1, v2 = b2 * v, (1 - b2) * g * g
    vv = v1 + v2
    dv = (3 * v1 + 4 * v2) * U + (1 - b2) * (2 * np.abs(g) * dg + dg * dg)
    r = np.sqrt(vv)
    with np.errstate(all="ignore"):
        dr = np.where(vv > 0, dv / (2 * np.maximum(r, 1e-300)), 0) + r * U
        den = r / np.sqrt(1 - b2 ** n) + eps
        dden = dr / np.sqrt(1 - b2 ** n) + (2 * r / np.sqrt(1 - b2 ** n) + 2 * eps + r) * U + den * U
        u = mm / den
        du = dm / den + np.abs(u) * (dden / den) + np.abs(u) * U
    s = lr / (1 - b1 ** n)
    t1, t2 = theta * (1 - decay * lr), s * u
    dt = np.abs(t1) * 4 * U + s * du + np.abs(t2) * 2 * U + (np.abs(t1) + np.abs(t2)) * U
    slack = 1.01             # products of the bounds themselves
    tiny = 2.0 ** -148       # results below the normal range
    return [(t1 - t2, dt * slack + tiny), (mm, dm * slack + tiny), (vv, dv * slack + tiny)]
