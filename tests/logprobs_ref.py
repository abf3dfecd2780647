"""Plain NumPy statements of token log probabilities for the tests: the binary32
definition step by step (the bits of the library), and binary64 with the rounding
errors of the former counted."""
import numpy as np

F32, F64 = np.float32, np.float64
P1, P2 = F32(float.fromhex("0x1.62e584p-1")), F32(float.fromhex("0x1.ebfbe0p-3"))
POWERS = np.exp2(np.arange(32) / 32).astype(F32).view(np.uint32).astype(np.int64)
LN2 = float.fromhex("0x1.62e42fefa39efp-1")
LOG2E = float.fromhex("0x1.71547652b82fep+0")
BLOCK, SEGMENT = 1024, 4096
U = 2.0 ** -24
E_REL = 2.3e-7      # of e for a given t: the fit's 5.3e-8, the power's and three roundings of at most 2^-24 each


def exp_t(x, m, c):
    """(e, t) of binary32 arrays x against m."""
    with np.errstate(all="ignore"):
        t = ((x - m).astype(F32) * c).astype(F32)
        t = np.where(np.isnan(t), t, np.maximum(t, F32(-127))).astype(F32)
        n = np.rint(F32(32) * t)
        f = (t - n / F32(32)).astype(F32)
        p = (((P2 * f).astype(F32) + P1) * f).astype(F32) + F32(1)
        n = np.where(np.isnan(n), 0, n).astype(np.int64)
        w = (POWERS[n % 32] + ((n // 32) << 23)).astype(np.uint32).view(F32)
        e = p * w
    return e.astype(F32), t


def halves(v):
    while v.shape[-1] > 1:
        h = v.shape[-1] // 2
        v = v[..., :h] + v[..., h:]
    return v[..., 0]


def ln_fixed(S):
    S = F32(S)
    if not S > 0:
        return F32(-np.inf) if S == 0 else S
    if not np.isfinite(S):
        return S
    F, E = np.frexp(S)          # F in [1/2, 1)
    F, E = F32(2) * F, F32(int(E) - 1)
    if F > F32(float.fromhex("0x1.6a09e6p+0")):
        F, E = F * F32(0.5), E + F32(1)
    z = (F - F32(1)) / (F + F32(1))
    zz, r = z * z, z + z
    p = F32(1 / 9)
    for n in (7, 5, 3):
        p = p * zz + F32(1 / n)
    ln_f = r + r * (zz * p)
    return E * F32(float.fromhex("0x1.62e400p-1")) + (ln_f + E * F32(float.fromhex("0x1.7f7d1cp-20")))


def segment(x, c):
    """(m, s, u) of up to 4096 columns."""
    M, s, u = F32(-np.inf), np.zeros(256, F32), np.zeros(256, F32)
    for b in range(0, len(x), BLOCK):
        p = np.full(BLOCK, -np.inf, F32)
        p[:len(x[b:b + BLOCK])] = x[b:b + BLOCK]
        to = F32(np.nan) if np.isnan(p).any() or np.isnan(M) else max(M, p.max())
        ref = F32(0) if to == -np.inf else to
        if not to == M:
            w, d = exp_t(np.array([M], F32), ref, c)
            u, s = w * (u + d * s), w * s
            M = to
        e, t = exp_t(p.reshape(4, 256), ref, c)
        for i in range(4):
            s, u = s + e[i], u + e[i] * t[i]
    return M, halves(s), halves(u)


def row(x, temperature):
    """(M, S, Q, ln S) of one row of binary32 logits."""
    c = F32(LOG2E / float(F32(temperature)))
    V = len(x)
    segs = -(-V // SEGMENT)
    m, s, u = (np.zeros(segs, F32) for _ in range(3))
    with np.errstate(all="ignore"):
        for j in range(segs):
            m[j], s[j], u[j] = segment(x[j * SEGMENT:(j + 1) * SEGMENT], c)
        M = F32(np.nan) if np.isnan(m).any() else m.max()
        w, tt = exp_t(m, F32(0) if M == -np.inf else M, c)
        S, Qs = np.zeros(32, F32), np.zeros(32, F32)
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
    inv = F32(1) / F32(temperature)
    out = [[] for _ in range(6)]
    for r, v in enumerate(x):
        M, S, Qs, ln = row(v, temperature)

        def logp(z):
            if z == -np.inf and M < np.inf:
                return F32(-np.inf)
            return (z - M) * inv - ln

        with np.errstate(all="ignore"):
            t = -1 if targets is None else int(targets[r])
            H = F32(0) if S == 0 else ln - F32(LN2) * (Qs / S)
            out[0].append(F32(0) if t < 0 else F32(np.nan) if t >= len(v) else logp(v[t]))
            out[1].append(M if S == 0 else M * inv + ln)
            out[2].append(H)
            out[3].append([M, F32(0) if S == 0 else F32(1) / S, ln, H])
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
                B = -(((inv * F32(LN2)) * dentropy[r]) * invS)
            A = -((inv * A) * invS)
            if M == -np.inf:
                A = B = G = F32(0)
            e, tt = exp_t(v, F32(0) if M == -np.inf else M, c)
            out[r] = e * (A + B * tt) if dentropy is not None else e * A
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
        # an exponential's error: of its argument (two roundings and the constant's) and of the
        # polynomial, each for the value, up to three raises of its segment's maximum and the row's;
        # the arguments add up to the value's; then 24 additions and four products, and in the row
        # four products and at most 10 additions
        rel = 5 * E_REL + az * 15 * U + 42 * U
        dS = (e * rel).sum(1) / S
        # q adds the rounding of t (as above) and of its products and sums
        dQ = (e * az * (rel + 15 * U + 50 * U)).sum(1) / S + (ez.sum(1) / S) * -dS + (e * 15 * U).sum(1) / S
        dln = dS + 6 * U * ln                   # the logarithm's own steps
    base = np.abs(M[:, 0] / temperature)
    out = {"lse": (M[:, 0] / temperature + ln, dln + 3 * U * base + U * np.abs(M[:, 0] / temperature + ln) + 1e-12),
           "entropy": (H, dln + dQ + 4 * U * (ln + np.abs(ez.sum(1) / S)) + 1e-12)}
    if targets is not None:
        t = np.clip(targets, 0, x.shape[1] - 1)
        zt = z[np.arange(len(x)), t]
        lp = zt - ln
        room = np.where(np.isinf(lp), 0, 3 * U * np.abs(np.where(np.isinf(zt), 0, zt)) + U * np.abs(np.where(np.isinf(lp), 0, lp)))
        out["logp"] = (np.where(targets < 0, 0, lp), dln + room + 1e-12)
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
    b = p * (np.abs(inner) * relp + mag * 8 * U + np.abs(h)[:, None] * (dH + dS + 6 * U * ln)[:, None]) / temperature
    rows = np.arange(len(x))
    on = targets >= 0
    g[rows[on], targets[on]] += w[on] / temperature
    b[rows[on], targets[on]] += np.abs(w[on]) / temperature * 3 * U
    return g, b * 1.01 + np.abs(g) * U + 2.0 ** -126
