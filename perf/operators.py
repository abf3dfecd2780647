"""Measured cases of the 8-bit and block-edge operators.

    gemm_i8                    matrix product of 8-bit integers with a scale for
                               each token (row of A) and channel (column of B)
    quantize_rows,             activation checkpoints in 8 bits: saved with a
    dequantize_rows            scale for every group of columns, and restored
    swiglu_backward_i8,        the backward pass read straight from such
    rmsnorm_backward_i8        checkpoints
    rmsnorm_residual           the norm after a block, its gate and residual
                               scale, the residual sum and the norm before the
                               next block, in one pass; and its backward

`run` computes a case in its plain form (elementary torch operations in
binary32), or through the library when `own` is true; `exact` computes it in
binary64.  Everything a case needs is made from its sizes and a seed.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
FLOOR = 2.0 ** -100      # the smallest magnitude a scale is taken from
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # W_o of a 2048-wide decoder layer for one token being generated
        {"name": "i8_token", "op": "gemm_i8", "M": 1, "N": 2048, "K": 2048, "out": "f32", "bias": False},
        # gate and up projections for the tokens of 13 sequences decoded together
        {"name": "i8_decode13", "op": "gemm_i8", "M": 13, "N": 16384, "K": 2048, "out": "bf16", "bias": False},
        # every size odd or just past a tile, rows of 3001 bytes, a bias
        {"name": "i8_ragged", "op": "gemm_i8", "M": 4097, "N": 1023, "K": 3001, "out": "f32", "bias": True},
        # gate and up projections of a whole 2048-token prompt
        {"name": "i8_prefill", "op": "gemm_i8", "M": 2048, "N": 16384, "K": 2048, "out": "f16", "bias": False},
        # the benchmark's square product
        {"name": "i8_square", "op": "gemm_i8", "M": 8192, "N": 8192, "K": 8192, "out": "bf16", "bias": False},
        # [g | u] of two 2048-token sequences kept for the backward pass and restored
        {"name": "ckpt_gate_up", "op": "checkpoint", "rows": 4096, "cols": 16384, "group": 128, "type": "f32"},
        # bfloat16 activations, one scale a token, an odd width
        {"name": "ckpt_token_odd", "op": "checkpoint", "rows": 4097, "cols": 1023, "group": 0, "type": "bf16"},
        # SwiGLU's backward of two sequences from the 8-bit [g | u], the activation recomputed for dW_down
        {"name": "swiglu_bwd", "op": "swiglu_backward", "rows": 4096, "cols": 8192, "group": 128},
        # the pre-norm's backward of two sequences, the residual gradient added, its output recomputed for dW
        {"name": "rmsnorm_bwd", "op": "rmsnorm_backward", "rows": 4096, "cols": 2048, "group": 128},
        # the edge between two blocks for one token being generated
        {"name": "edge_token", "op": "edge", "rows": 1, "cols": 2048, "post": True, "gates": 1, "alpha": 0.5},
        # the same for two 2048-token sequences, a gate for each
        {"name": "edge_fwd", "op": "edge", "rows": 4096, "cols": 2048, "post": True, "gates": 2, "alpha": 0.5},
        # its backward over a larger batch
        {"name": "edge_bwd", "op": "edge_backward", "rows": 8192, "cols": 2048, "post": True, "gates": 1,
         "alpha": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm_i8", "gemm_i8", "checkpoint", "swiglu_backward", "rmsnorm_backward", "edge",
                     "edge_backward"])
    if op == "gemm_i8":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 16384), "K": _log(rng, 64, 4096),
                "out": rng.choice(["f32", "f16", "bf16"]), "bias": rng.random() < 0.5}
    if op == "checkpoint":
        return {"op": op, "rows": _log(rng, 1, 4096), "cols": _log(rng, 32, 16384),
                "group": rng.choice([0, 32, 64, 128, 256]), "type": rng.choice(["f32", "f16", "bf16"])}
    if op == "swiglu_backward":
        return {"op": op, "rows": _log(rng, 1, 4096), "cols": _log(rng, 32, 8192),
                "group": rng.choice([0, 32, 64, 128, 256])}
    if op == "rmsnorm_backward":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 32, 8192),
                "group": rng.choice([0, 32, 64, 128, 256])}
    gates = rng.choice([0, 1, 3])
    rows = _log(rng, 1, 8192)
    if gates > 1:
        rows = max(1, rows // gates) * gates
    return {"op": op, "rows": rows, "cols": _log(rng, 32, 8192), "post": rng.random() < 0.7, "gates": gates,
            "alpha": rng.choice([1.0, 0.5, 0.17])}


# ----------------------------------------------------------------- inputs ----

def _ngroups(cols, group):
    return -(-cols // group) if group else 1


def _quantize(x, group):
    """(whole numbers, scales) of rows of x in the format of quantize_rows:
    for every group amax, a = max(amax, 2^-100), scale = a / 127,
    q = rint(x * (127 / a)); every step one binary32 rounding."""
    rows, cols = x.shape
    n = _ngroups(cols, group)
    width = group if group else cols
    xp = torch.nn.functional.pad(x.float(), (0, n * width - cols)).view(rows, n, width)
    a = xp.abs().amax(2).clamp_min(FLOOR)
    c127 = torch.full_like(a, 127.0)
    scale = torch.div(a, c127)
    q = torch.round(xp * torch.div(c127, a).unsqueeze(2))
    ok = torch.isfinite(a)
    scale = torch.where(ok, scale, torch.full_like(scale, float("nan")))
    q = torch.where(ok.unsqueeze(2), q, torch.zeros_like(q))
    return q.view(rows, n * width)[:, :cols].to(torch.int8).contiguous(), scale


def _spread(scale, cols, group):
    """Each column's scale."""
    return scale.repeat_interleave(group, 1)[:, :cols] if group else scale.expand(-1, cols)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op == "gemm_i8":
        st["A"], s = _quantize(_randn(g, case["M"], case["K"]), 0)
        st["a_scale"] = s.view(-1)
        st["W"], s = _quantize(_randn(g, case["N"], case["K"]) * 0.02, 0)
        st["b_scale"] = s.view(-1)
        st["bias"] = _randn(g, case["N"]) * 0.02 if case["bias"] else None
    elif op == "checkpoint":
        st["x"] = _randn(g, case["rows"], case["cols"]).to(DTYPES[case["type"]])
    elif op == "swiglu_backward":
        r, c = case["rows"], case["cols"]
        st["g"], st["gs"] = _quantize(_randn(g, r, c) * 2.0, case["group"])
        st["u"], st["us"] = _quantize(_randn(g, r, c) * 2.0, case["group"])
        st["dh"] = _randn(g, r, c) * 1e-2
    elif op == "rmsnorm_backward":
        r, c = case["rows"], case["cols"]
        st["x"], st["xs"] = _quantize(_randn(g, r, c), case["group"])
        st["gamma"] = 1.0 + 0.1 * _randn(g, c)
        st["dy"] = _randn(g, r, c) * 1e-2
        st["res"] = _randn(g, r, c) * 1e-2
    else:
        r, c = case["rows"], case["cols"]
        st["x"] = _randn(g, r, c)
        st["f"] = _randn(g, r, c) * 3.0
        st["pre"] = 1.0 + 0.1 * _randn(g, c)
        st["post"] = 1.0 + 0.1 * _randn(g, c) if case["post"] else None
        st["gate"] = 0.5 + 0.2 * _randn(g, case["gates"], c) if case["gates"] else None
        if op == "edge_backward":
            # the forward's output, and the gradients of both of its results
            st["y"] = st.pop("x") + case["alpha"] * st["f"]
            st["dy"] = _randn(g, r, c) * 1e-2
            st["dh"] = _randn(g, r, c) * 1e-2
    return st


# -------------------------------------------------------------- the passes ----

def _run_own(st):
    import verifiable_repops_gemm_gb300 as rp
    case = st["case"]
    op = case["op"]
    if op == "gemm_i8":
        return rp.gemm_i8(st["A"], st["W"].t(), st["a_scale"], st["b_scale"], out_dtype=DTYPES[case["out"]],
                          bias=st["bias"])
    if op == "checkpoint":
        q, s = rp.quantize_rows(st["x"], group=case["group"])
        return rp.dequantize_rows(q, s, group=case["group"]), s
    if op == "swiglu_backward":
        h = torch.empty_like(st["dh"])
        dg, du = rp.swiglu_backward_i8(st["g"], st["gs"], st["u"], st["us"], st["dh"], group=case["group"], h=h)
        return dg, du, h
    if op == "rmsnorm_backward":
        h = torch.empty_like(st["dy"])
        dx, dgamma = rp.rmsnorm_backward_i8(st["x"], st["xs"], st["gamma"], EPS, st["dy"], group=case["group"],
                                            res=st["res"], h=h)
        return dx, dgamma, h
    if op == "edge":
        return rp.rmsnorm_residual(st["x"], st["f"], st["pre"], EPS, post_gain=st["post"], gate=st["gate"],
                                   alpha=case["alpha"])
    out = rp.rmsnorm_residual_backward(st["dy"], st["dh"], st["y"], st["f"], st["pre"], EPS, post_gain=st["post"],
                                       gate=st["gate"], alpha=case["alpha"])
    return tuple(t for t in out if t is not None)


def _rms_inv(x):
    return torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)


def _rows_of(gate, rows):
    return gate.repeat_interleave(rows // gate.shape[0], 0)


def _rmsnorm_backward(x, gamma, dy):
    """(dx, dy * xhat) of y = xhat * gamma."""
    inv = _rms_inv(x)
    xh = x * inv
    gy = dy * gamma
    return inv * (gy - xh * (gy * xh).mean(1, keepdim=True)), dy * xh


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "gemm_i8":
        y = (st["A"].float() @ st["W"].t().float()) * st["a_scale"][:, None] * st["b_scale"]
        if st["bias"] is not None:
            y = y + st["bias"]
        return y.to(DTYPES[case["out"]])
    if op == "checkpoint":
        q, s = _quantize(st["x"], case["group"])
        return q.float() * _spread(s, case["cols"], case["group"]), s
    if op == "swiglu_backward":
        c = case["cols"]
        g = st["g"].float() * _spread(st["gs"], c, case["group"])
        u = st["u"].float() * _spread(st["us"], c, case["group"])
        sg = 1.0 / (1.0 + torch.exp(-g))
        silu = g * sg
        return st["dh"] * u * (sg * (1.0 + g * (1.0 - sg))), st["dh"] * silu, silu * u
    if op == "rmsnorm_backward":
        x = st["x"].float() * _spread(st["xs"], case["cols"], case["group"])
        dx, p = _rmsnorm_backward(x, st["gamma"], st["dy"])
        return dx + st["res"], p.sum(0), x * _rms_inv(x) * st["gamma"]
    f, alpha = st["f"], case["alpha"]
    if op == "edge":
        p = f if st["post"] is None else f * _rms_inv(f) * st["post"]
        if st["gate"] is not None:
            p = p * _rows_of(st["gate"], case["rows"])
        y = st["x"] + alpha * p
        return y, y * _rms_inv(y) * st["pre"]
    d, pp = _rmsnorm_backward(st["y"], st["pre"], st["dh"])
    dx = d + st["dy"]
    dt = alpha * dx
    p = f if st["post"] is None else f * _rms_inv(f) * st["post"]
    dp = dt if st["gate"] is None else dt * _rows_of(st["gate"], case["rows"])
    out = [dx]
    if st["post"] is None:
        out += [dp, pp.sum(0)]
    else:
        df, q = _rmsnorm_backward(f, st["post"], dp)
        out += [df, pp.sum(0), q.sum(0)]
    if st["gate"] is not None:
        out.append((dt * p).view(st["gate"].shape[0], -1, case["cols"]).sum(1))
    return tuple(out)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- work ----

def work(case):
    op = case["op"]
    if op == "gemm_i8":
        M, N, K = case["M"], case["N"], case["K"]
        b = M * K + N * K + 4 * (M + N) + SIZE[case["out"]] * M * N + (4 * N if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * M * N * K}
    n = case["rows"] * case["cols"]
    if op == "checkpoint":
        s = 4 * case["rows"] * _ngroups(case["cols"], case["group"])
        # x in; the whole numbers and scales written; the restored values out
        return {"bytes": n * (SIZE[case["type"]] + 1 + 4) + s, "flops": 4 * n}
    if op == "swiglu_backward":
        s = 4 * case["rows"] * _ngroups(case["cols"], case["group"])
        return {"bytes": n * (2 + 4 + 12) + 2 * s, "flops": 15 * n}
    if op == "rmsnorm_backward":
        s = 4 * case["rows"] * _ngroups(case["cols"], case["group"])
        return {"bytes": n * (1 + 8 + 8) + s + 8 * case["cols"], "flops": 15 * n}
    vec = 4 * case["cols"]
    if op == "edge":
        return {"bytes": 16 * n + vec * (1 + int(case["post"]) + case["gates"]), "flops": 12 * n}
    return {"bytes": 24 * n + 2 * vec * (1 + int(case["post"]) + case["gates"]), "flops": 30 * n}


# ------------------------------------------------------------------ exact ----

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    D = torch.float64
    if op == "gemm_i8":
        acc = torch.matmul(st["A"].to(D), st["W"].to(D).T)      # whole numbers below 2^53
        acc *= st["a_scale"].to(D).unsqueeze(1)
        acc *= st["b_scale"].to(D).unsqueeze(0)
        return acc if st["bias"] is None else acc + st["bias"].to(D)
    if op == "checkpoint":
        # scale and 127 / a are binary32 values by the format's definition (a
        # binary64 quotient of binary32 values rounds to the same one)
        x = st["x"].to(D)
        cols, width = case["cols"], case["group"] or case["cols"]
        vals, scales = torch.empty_like(x), []
        for j in range(0, cols, width):
            part = x[:, j:j + width]
            a = part.abs().max(dim=1, keepdim=True).values.clamp(min=FLOOR)
            s = (a / 127.0).float().to(D)
            q = torch.round((part * (127.0 / a).float().to(D)).float().to(D))
            vals[:, j:j + width] = q * s
            scales.append(s)
        return vals, torch.cat(scales, dim=1)

    def wide(q, s):
        cols = q.shape[1]
        idx = torch.arange(cols, device=q.device) // (case["group"] or cols)
        return q.to(D) * s.to(D)[:, idx]

    def norm(v, gain):
        r = (v.square().sum(1) / v.shape[1] + EPS).sqrt().unsqueeze(1)
        return v / r, r, v / r * gain.to(D)

    def norm_grad(v, gain, d):
        vh, r, _ = norm(v, gain)
        t = d * gain.to(D)
        return (t - vh * ((t * vh).sum(1) / v.shape[1]).unsqueeze(1)) / r, (d * vh).sum(0)

    if op == "swiglu_backward":
        g, u, dh = wide(st["g"], st["gs"]), wide(st["u"], st["us"]), st["dh"].to(D)
        s = torch.sigmoid(g)
        return dh * u * (s + g * s * (1.0 - s)), dh * g * s, g * s * u
    if op == "rmsnorm_backward":
        x = wide(st["x"], st["xs"])
        dx, dgamma = norm_grad(x, st["gamma"], st["dy"].to(D))
        return dx + st["res"].to(D), dgamma, norm(x, st["gamma"])[2]
    f, alpha, rows = st["f"].to(D), case["alpha"], case["rows"]
    gate = 1.0
    if st["gate"] is not None:
        G = st["gate"].shape[0]
        gate = st["gate"].to(D)[torch.arange(rows, device=f.device) // (rows // G)]
    p = f if st["post"] is None else norm(f, st["post"])[2]
    if op == "edge":
        y = st["x"].to(D) + alpha * gate * p
        return y, norm(y, st["pre"])[2]
    d, dpre = norm_grad(st["y"].to(D), st["pre"], st["dh"].to(D))
    dx = d + st["dy"].to(D)
    dp = alpha * gate * dx
    if st["post"] is None:
        out = [dx, dp, dpre]
    else:
        df, dpost = norm_grad(f, st["post"], dp)
        out = [dx, df, dpre, dpost]
    if st["gate"] is not None:
        out.append(torch.stack([t.sum(0) for t in (alpha * dx * p).split(rows // st["gate"].shape[0])]))
    return tuple(out)
