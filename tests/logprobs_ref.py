"""Plain NumPy statements of token log probabilities for the tests: the binary32
definition step by step (the bits of the library), and binary64 with the rounding
errors of the former counted."""
import numpy as np

F32, F64 = np.float32, np.float64
Q = [F32(float.fromhex(h)) for h in ("0x1.5bba14p-10", "0x1.3cea88p-7", "0x1.c6b752p-5", "0x1.ebf9bcp-3",
                                     "0x1.62e42ap-1")] + [F32(1)]
LN2 = float.fromhex("0x1.62e42fefa39efp-1")
LOG2E = float.fromhex("0x1.71547652b82fep+0")
SEGMENT = 1024
U = 2.0 ** -24
E_REL = 2.0e-7      # of p: the fit's 9.2e-8, its coefficients' and Horner's roundings (measured 1.9e-7)


def exp_t(x, m, c):
    """(e, t) of binary32 arrays x against m."""
    with np.errstate(all="ignore"):
        t = ((x - m).astype(F32) * c).astype(F32)
        t = np.where(np.isnan(t), t, np.maximum(t, F32(-127))).astype(F32)
        k = np.rint(t)
        f = (t - k).astype(F32)
        p = np.full_like(f, Q[0])
        for q in Q[1:]:
            p = (p * f).astype(F32) + q
        e = np.where(k <= -127, F32(0) * p, np.ldexp(p, np.where(np.isnan(k), 0, k).astype(np.int32)))
    return e.astype(F32), t


def halves(v):
    while v.shape[-1] > 1:
        h = v.shape[-1] // 2
        v = v[..., :h] + v[..., h:]
    return v[..., 0]


def ln_fixed(S):
    if not S > 0:
        return -np.inf if S == 0 else S
    F, E = np.frexp(S)          # F in [1/2, 1)
    F, E = 2 * F, int(E) - 1
    if F > 1.41421356237309504880:
        F, E = F / 2, E + 1
    z = (F - 1) / (F + 1)
    zz = z * z
    p = 1.0 / 23
    for n in range(10, -1, -1):
        p = p * zz + 1.0 / (2 * n + 1)
    return E * LN2 + (2 * z) * p


def row(x, temperature):
    """(M, S, Q, ln S) of one row of binary32 logits."""
    c = F32(LOG2E / float(F32(temperature)))
    V = len(x)
    segs = -(-V // SEGMENT)
    pad = np.full(segs * SEGMENT, -np.inf, F32)
    pad[:V] = x
    parts = pad.reshape(segs, SEGMENT)
    m = np.array([np.nan if np.isnan(p).any() else p.max() for p in parts], F32)
    ref = np.where(m == -np.inf, F32(0), m)
    e, t = exp_t(parts, ref[:, None], c)
    with np.errstate(all="ignore"):
        s = np.zeros((segs, 256), F32)
        u = np.zeros((segs, 256), F32)
        for i in range(4):
            s = s + e[:, 256 * i:256 * i + 256]
            u = u + e[:, 256 * i:256 * i + 256] * t[:, 256 * i:256 * i + 256]
        s, u = halves(s), halves(u)
        M = F32(np.nan) if np.isnan(m).any() else m.max()
        w, tt = exp_t(m, F32(0) if M == -np.inf else M, c)
        w, tt, s, u = (a.astype(F64) for a in (w, tt, s, u))
        S, Qs = np.zeros(32), np.zeros(32)
        for j in range(segs):
            S[j % 32] += w[j] * s[j]
            Qs[j % 32] += w[j] * (u[j] + tt[j] * s[j])
        S, Qs = halves(S), halves(Qs)
    return M, S, Qs, ln_fixed(S)


def order(x):
    """Columns by falling value, NaN first, the lower column first among equals."""
    key = np.where(np.isnan(x), np.inf, x).astype(F64)
    return np.lexsort((np.arange(len(x)), -key, ~np.isnan(x)))


def forward(x, targets, temperature, top):
    """The library's results, bit for bit: logp, lse, entropy, stats, top_logp, top_ids."""
    inv = 1.0 / float(F32(temperature))
    out = [[] for _ in range(6)]
    for r, v in enumerate(x):
        M, S, Qs, ln = row(v, temperature)

        def logp(z):
            if z == -np.inf and M < np.inf:
                return F32(-np.inf)
            return F32((F64(z) - F64(M)) * inv - ln)

        with np.errstate(all="ignore"):
            t = -1 if targets is None else int(targets[r])
            H = F32(0) if S == 0 else F32(ln - LN2 * (Qs / S))
            out[0].append(F32(0) if t < 0 else F32(np.nan) if t >= len(v) else logp(v[t]))
            out[1].append(M if S == 0 else F32(F64(M) * inv + ln))
            out[2].append(H)
            out[3].append([M, F32(0) if S == 0 else F32(1 / S), F32(ln), H])
            ids = order(v)[:top]
            out[4].append([logp(v[i]) for i in ids])
            out[5].append(ids)
    n = len(x)
    return [np.array(out[0], F32), np.array(out[1], F32), np.array(out[2], F32), np.array(out[3], F32).reshape(n, 4),
            np.array(out[4], F32).reshape(n, top), np.array(out[5], np.int64).reshape(n, top)]


def backward(x, targets, stats, dlogp, dentropy, temperature):
    """The gradient in binary32 before it is narrowed, bit for bit."""
    c, inv = F32(LOG2E / float(F32(temperature))), F32(1) / F32(temperature)
    out = np.empty(x.shape, F32)
    with np.errstate(all="ignore"):
        for r, v in enumerate(x):
            M, invS, ln, H = stats[r]
            t = -1 if targets is None else int(targets[r])
            w = F32(0) if t < 0 or dlogp is None else dlogp[r]
            if t >= len(v) and dlogp is not None:
                w = F32(np.nan)
            A, B, G = w, F32(0), inv * w
            if dentropy is not None:
                A = A + dentropy[r] * (H - ln)
                B = -((inv * F32(LN2)) * dentropy[r])
            A = -(inv * A)
            if M == -np.inf:
                A = B = G = F32(0)
            e, tt = exp_t(v, F32(0) if M == -np.inf else M, c)
            p = e * invS
            out[r] = p * (A + B * tt) if dentropy is not None else p * A
            if 0 <= t < len(v):
                out[r, t] = out[r, t] + G
    return out


def forward64(x, targets, temperature):
    """{name: (value, bound)} of logp, lse, entropy and the matrices z and ln p for
    finite-or--inf rows with something possible, in binary64."""
    temperature = float(F32(temperature))
    x = x.astype(F64)
    M = x.max(1, keepdims=True)
    with np.errstate(all="ignore"):
        z = (x - M) / temperature
        e = np.exp(z)
        S = e.sum(1)
        ln = np.log(S)
        ez = np.where(e > 0, e * z, 0)
        H = ln - ez.sum(1) / S
        az = np.where(e > 0, -z, 0)
        # an exponential's error: of its argument (two roundings and the constant's, twice: against
        # the segment's maximum and that against the row's) and of the polynomial (twice); then 12
        # additions and a product
        rel = 2 * E_REL + az * 6 * U + 16 * U
        dS = (e * rel).sum(1) / S
        # q adds the rounding of t (as above) and of its product and sums
        dQ = (e * az * (rel + 6 * U + 16 * U)).sum(1) / S + (ez.sum(1) / S) * -dS + (e * 6 * U).sum(1) / S
    out = {"lse": (M[:, 0] / temperature + ln, dS + U * np.abs(M[:, 0] / temperature + ln) + 1e-12),
           "entropy": (H, dS + dQ + U * np.abs(H) + 1e-12)}
    if targets is not None:
        t = np.clip(targets, 0, x.shape[1] - 1)
        lp = z[np.arange(len(x)), t] - ln
        out["logp"] = (np.where(targets < 0, 0, lp), dS + U * np.abs(np.where(np.isinf(lp), 0, lp)) + 1e-12)
    return out, z, e, S, ln, H, dS


def backward64(x, targets, dlogp, dentropy, temperature):
    """(value, bound) of the gradient in binary64."""
    temperature = float(F32(temperature))
    _, z, e, S, ln, H, dS = forward64(x, targets, temperature)
    f, _, _, _, _, _, _ = forward64(x, targets, temperature)
    dH = f["entropy"][1]
    p = e / S[:, None]
    with np.errstate(all="ignore"):
        lp = np.where(p > 0, z - ln[:, None], 0)
        az = np.where(e > 0, -z, 0)
    w = np.where(targets < 0, 0, dlogp).astype(F64) if dlogp is not None else np.zeros(len(x))
    h = dentropy.astype(F64) if dentropy is not None else np.zeros(len(x))
    inner = w[:, None] + h[:, None] * (lp + H[:, None])
    g = -p * inner / temperature
    mag = np.abs(w)[:, None] + np.abs(h)[:, None] * (az + np.abs(ln)[:, None] + H[:, None])
    relp = E_REL + az * 3 * U + dS[:, None] + 4 * U
    b = p * (np.abs(inner) * relp + mag * 8 * U + np.abs(h)[:, None] * (dH + dS)[:, None]) / temperature
    rows = np.arange(len(x))
    on = targets >= 0
    g[rows[on], targets[on]] += w[on] / temperature
    b[rows[on], targets[on]] += np.abs(w[on]) / temperature * 3 * U
    return g, b * 1.01 + np.abs(g) * U + 2.0 ** -126
