"""Measured cases of the operators at the ends of a language model's training
step: positions, loss and update.

    token_logprobs,            log probabilities of given tokens with entropy and
    token_logprobs_backward    the top alternatives, and the gradient of the logits
    head_norm_rope,            norms of the query and key heads with the position
    head_norm_rope_backward    rotation in the same pass (adjacent pairs or halves,
                               all of a head or its first part), and the gradients
    adamw, adamw_moments       an AdamW step over many tensors at once, from one or
                               several contributors' gradients, with moments in 32
                               bits or in 8

`run` computes a case in its plain form (elementary torch operations in
binary32), or through the library when `own` is true; `exact` computes it in
binary64.  Everything a case needs is made from its sizes and a seed.
"""
import functools
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
GROUP = 128              # elements that share a scale in 8-bit moments
ADAM = {"lr": 3e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "decay": 0.1}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one token being generated: its log probability and 8 alternatives
        {"name": "lp_token", "op": "logprobs", "M": 1, "V": 131072, "type": "f32", "top": 8, "temp": 1.0},
        # 48 sequences decoded together, an odd vocabulary, sampled at a temperature
        {"name": "lp_decode48", "op": "logprobs", "M": 48, "V": 50021, "type": "bf16", "top": 20, "temp": 0.7},
        # scoring two 2048-token answers
        {"name": "lp_score", "op": "logprobs", "M": 4096, "V": 131072, "type": "bf16", "top": 1, "temp": 1.0},
        # the loss and its gradient for two 2048-token sequences
        {"name": "lp_train", "op": "logprobs_train", "M": 4096, "V": 32768, "type": "f32", "entropy": False},
        # the same with an entropy bonus, half-precision logits, a larger vocabulary
        {"name": "lp_train_entropy", "op": "logprobs_train", "M": 2048, "V": 131072, "type": "bf16", "entropy": True},
        # one token being generated far into a long context
        {"name": "qk_token", "op": "qk", "rows": 1, "q": 32, "k": 8, "dim": 64, "rot": 64, "layout": "adjacent",
         "type": "f32", "table": 131072},
        # two 2048-token prompts of a 2048-wide decoder layer
        {"name": "qk_prefill", "op": "qk", "rows": 4096, "q": 32, "k": 8, "dim": 64, "rot": 64, "layout": "adjacent",
         "type": "f32", "table": 2048},
        # a padded batch, heads of 80 of which 32 values are rotated
        {"name": "qk_ragged", "op": "qk", "rows": 4099, "q": 12, "k": 3, "dim": 80, "rot": 32, "layout": "halves",
         "type": "bf16", "table": 4096},
        # the backward pass of qk_prefill
        {"name": "qk_bwd", "op": "qk_backward", "rows": 4096, "q": 32, "k": 8, "dim": 64, "rot": 64,
         "layout": "adjacent", "type": "f32", "table": 2048},
        # gains, biases and gates: 200 tensors, the smallest of one value
        {"name": "adam_small", "op": "adamw", "tensors": 200, "most": 8192, "bits": 32, "grads": 1, "type": "f32"},
        # a 2048-wide decoder layer's weights
        {"name": "adam_layer", "op": "adamw", "tensors": 0, "most": 8192, "bits": 32, "grads": 1, "type": "f32"},
        # the same from four contributors' half-precision gradients, moments in 8 bits and restored
        {"name": "adam_layer8", "op": "adamw", "tensors": 0, "most": 8192, "bits": 8, "grads": 4, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_train", "qk", "qk_backward", "adamw", "adamw"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op.startswith("logprobs"):
        V = _log(rng, 100, 131072)
        M = _log(rng, 1, min(4096, (1 << 28) // V))
        if op == "logprobs":
            return {"op": op, "M": M, "V": V, "type": kind, "top": rng.choice([0, 1, 5, 20, 32]),
                    "temp": rng.choice([1.0, 0.7, 1.3])}
        return {"op": op, "M": M, "V": V, "type": kind, "entropy": rng.random() < 0.5}
    if op.startswith("qk"):
        dim = rng.choice([32, 64, 80, 96, 128, 256])
        k = rng.choice([1, 2, 3, 4, 8])
        return {"op": op, "rows": _log(rng, 1, 4096), "q": k * rng.choice([1, 2, 3, 4]), "k": k, "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2, 2 * (dim // 8)]), "layout": rng.choice(["adjacent", "halves"]),
                "type": kind, "table": rng.choice([4096, 65536])}
    return {"op": op, "tensors": _log(rng, 1, 400), "most": _log(rng, 16, 200000), "bits": rng.choice([32, 8]),
            "grads": rng.choice([1, 1, 3]), "type": kind}


# ----------------------------------------------------------------- inputs ----

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _sizes(case):
    """The tensors' sizes of an AdamW case and whether each is decayed."""
    if case["tensors"] == 0:                 # norms, qkv, output, gate and up, down
        d, f = 2048, case["most"]
        return [d, d * (d + 1024), d * d, d, 2 * d * f, f * d], [False, True, True, False, True, True]
    r = random.Random(case["tensors"] * 1000003 + case["most"])
    n = [1] + [max(1, int(math.exp(r.uniform(0.0, math.log(case["most"]))))) for _ in range(case["tensors"] - 1)]
    return n, [r.random() < 0.5 for _ in n]


def _slots(sizes):
    """Each tensor's offset in a flat buffer, on a multiple of GROUP, and its length."""
    out, at = [], 0
    for n in sizes:
        out.append(at)
        at += -(-n // GROUP) * GROUP
    return out, at


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    dt = DTYPES.get(case["type"])
    if op.startswith("logprobs"):
        M, V = case["M"], case["V"]
        x = torch.empty(M, V, dtype=dt, device=DEV)
        step = max(1, (1 << 26) // V)
        for r in range(0, M, step):          # a few likely tokens above the others
            part = _randn(g, min(step, M - r), V)
            x[r:r + step] = part * 2.0 + (part > 3.0) * part * 1.5
        x[:, V - V // 100:] = -math.inf      # the vocabulary's padding
        st["logits"] = x
        t = torch.randint(0, V - V // 100, (M,), generator=g, device=DEV)
        if M > 8:
            t[M // 7] = -100                 # a token without a target
        st["targets"] = t
        if op == "logprobs_train":
            st["dlogp"] = -(0.5 + torch.rand(M, generator=g, device=DEV)) / M
            st["dentropy"] = torch.full((M,), -0.01 / M, device=DEV) if case["entropy"] else None
    elif op.startswith("qk"):
        rows, heads, dim, pairs = case["rows"], case["q"] + case["k"], case["dim"], case["rot"] // 2
        # a block of the columns of a wider matrix: the values' heads follow
        st["x"] = (_randn(g, rows, (heads + case["k"]) * dim) * 1.5).to(dt)[:, :heads * dim]
        st["q_gain"] = 1.0 + 0.1 * _randn(g, dim)
        st["k_gain"] = 1.0 + 0.1 * _randn(g, dim)
        freq = torch.exp(torch.arange(pairs, device=DEV, dtype=torch.float64) * (-math.log(500000.0) / pairs)).float()
        angle = torch.arange(case["table"], device=DEV, dtype=torch.float64)[:, None] * freq.double()
        st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
        pos = torch.randint(0, case["table"], (rows,), generator=g, device=DEV, dtype=torch.int32)
        if rows > 8:
            pos[rows - rows // 9:] = -1      # the batch's padding
        st["pos"] = pos
        if op == "qk_backward":
            st["dy"] = (_randn(g, rows, heads * dim) * 1e-2).to(dt)
        st["out"] = torch.zeros(rows, heads * dim, dtype=dt, device=DEV)
    else:
        sizes, decayed = _sizes(case)
        at, total = _slots(sizes)
        st["sizes"], st["at"] = sizes, at
        lengths = torch.tensor([b - a for a, b in zip(at, at[1:] + [total])], device=DEV)
        tensor = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), lengths)
        live = torch.arange(total, device=DEV) - torch.tensor(at, device=DEV)[tensor] < \
            torch.tensor(sizes, device=DEV)[tensor]
        st["lengths"] = lengths
        st["theta"] = _randn(g, total) * 0.02 * live
        # gradients whose size differs from tensor to tensor and from row to row
        size = torch.exp(_randn(g, len(sizes)))[tensor] * torch.exp(_randn(g, total // GROUP)).repeat_interleave(GROUP)
        st["grads"] = [(_randn(g, total) * 1e-3 * size * live).to(dt) for _ in range(case["grads"])]
        st["decay"] = [ADAM["decay"] if d else 0.0 for d in decayed]
        m = _randn(g, total) * 3e-4 * size * live
        v = (1e-3 * size).square() * (0.5 + torch.rand(total, generator=g, device=DEV)) * live
        if case["bits"] == 32:
            st["m"], st["v"] = m, v
        else:
            seeds = torch.zeros(total, dtype=torch.int64, device=DEV)
            (st["m"], st["m_scale"]), (st["v"], st["v_scale"]) = _encode(m, 3, seeds), _encode(v.sqrt(), 4, seeds)
        st["step"] = 100

        def views(flat, per=1):
            return [flat[a // per:a // per + -(-n // per)] for a, n in zip(at, sizes)]

        st["views"] = {k: views(st[k]) for k in ("theta", "m", "v")}
        st["views"]["grads"] = [views(t) for t in st["grads"]]
        if case["bits"] == 8:
            st["views"].update({k: views(st[k], GROUP) for k in ("m_scale", "v_scale")})
    return st


# -------------------------------------------------------------- the passes ----

def _run_own(st):
    import verifiable_repops_gemm_gb300 as rp
    case = st["case"]
    op = case["op"]
    if op == "logprobs":
        r = rp.token_logprobs(st["logits"], st["targets"], temperature=case["temp"], top=case["top"])
        return (r.logp, r.lse, r.entropy) + ((r.top_logp, r.top_ids) if case["top"] else ())
    if op == "logprobs_train":
        r = rp.token_logprobs(st["logits"], st["targets"])
        d = rp.token_logprobs_backward(st["logits"], st["targets"], r.stats, st["dlogp"], st["dentropy"])
        return r.logp, r.lse, r.entropy, d
    if op == "qk":
        return rp.head_norm_rope(st["x"], case["q"], case["k"], st["cos"], st["sin"], q_gain=st["q_gain"],
                                 k_gain=st["k_gain"], eps=EPS, layout=case["layout"], positions=st["pos"],
                                 out=st["out"])
    if op == "qk_backward":
        return rp.head_norm_rope_backward(st["dy"], st["x"], case["q"], case["k"], st["cos"], st["sin"],
                                          q_gain=st["q_gain"], k_gain=st["k_gain"], eps=EPS, layout=case["layout"],
                                          positions=st["pos"], dx=st["out"])
    v = st["views"]
    more = {"m_scales": v["m_scale"], "v_scales": v["v_scale"]} if case["bits"] == 8 else {}
    rp.adamw(v["theta"], v["grads"], v["m"], v["v"], step=st["step"], lr=ADAM["lr"],
             betas=(ADAM["beta1"], ADAM["beta2"]), eps=ADAM["eps"], weight_decay=st["decay"], **more)
    if case["bits"] == 32:
        return st["theta"], st["m"], st["v"]
    return (st["theta"],) + rp.adamw_moments(st["m"], st["v"], st["m_scale"], st["v_scale"])


def _ordered(x):
    """Whole numbers in the order of a binary32 matrix's values, the lower column first among equals."""
    b = (x + 0.0).view(torch.int32).to(torch.int64)
    b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
    return b * (1 << 31) + (torch.arange(x.shape[1], 0, -1, device=x.device) - 1)


def _logprobs(st, temp, top):
    x, t = st["logits"].float(), st["targets"]
    m = x.amax(1, keepdim=True)
    z = (x - m) * (1.0 / temp)
    e = torch.exp(z)
    total = e.sum(1)
    log = torch.log(total)
    entropy = log - torch.where(e > 0, e * z, torch.zeros_like(e)).sum(1) / total
    logp = torch.gather(z, 1, t.clamp_min(0)[:, None])[:, 0] - log
    out = [torch.where(t < 0, torch.zeros_like(logp), logp), m[:, 0] * (1.0 / temp) + log, entropy]
    if top:
        key = torch.topk(_ordered(x), top, 1).values
        ids = x.shape[1] - 1 - torch.remainder(key, 1 << 31)
        out += [torch.gather(z, 1, ids) - log[:, None], ids]
    return out, z, e, total, log


def _logprobs_gradient(st, entropy, z, e, total, log):
    t = st["targets"]
    w = torch.where(t < 0, torch.zeros_like(st["dlogp"]), st["dlogp"])[:, None]
    p = e / total[:, None]
    d = -p * w
    if st["dentropy"] is not None:
        lp = torch.where(p > 0, z - log[:, None], torch.zeros_like(p))
        d = d - st["dentropy"][:, None] * p * (lp + entropy[:, None])
    return d.scatter_add_(1, t.clamp_min(0)[:, None], w).to(st["logits"].dtype)


def _by_head(st, name):
    case = st["case"]
    return st[name].float().view(case["rows"], case["q"] + case["k"], case["dim"])


def _gains(st):
    """Each head's gain."""
    case = st["case"]
    return torch.cat([st["q_gain"].expand(case["q"], -1), st["k_gain"].expand(case["k"], -1)])


def _rotate(st, x, sign):
    """The first columns of every head rotated to each row's position, or back (sign -1)."""
    case = st["case"]
    pairs = case["rot"] // 2
    pos = st["pos"].clamp_min(0).long()
    c, s = st["cos"][pos][:, None], st["sin"][pos][:, None] * sign
    if case["layout"] == "adjacent":
        a, b = x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
        y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = x[..., :pairs], x[..., pairs:2 * pairs]
        y = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([y, x[..., 2 * pairs:]], -1)


def _unpadded(st, y):
    """y's rows where a row has a position, the output's own elsewhere."""
    y = y.flatten(1).to(st["out"].dtype)
    return torch.where(st["pos"][:, None] >= 0, y, st["out"])


def _mix(h):
    """The finaliser of MurmurHash3 (Appleby) on 32-bit values held in 64."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _encode(x, bits, dither):
    """(codes, scales): a sign (3 bits of mantissa) or none (4), 4 bits of exponent, and `bits` of
    mantissa, in units of a power of two for each group; rounded up with the probability that `dither`
    (16 bits) has of passing what is cut off."""
    shift = 23 - bits
    most = 0x600000 if bits == 3 else 0x780000            # 1.75 and 1.9375: the largest code
    unit = 8 if bits == 3 else 0
    amax = x.abs().view(-1, GROUP).amax(1).view(torch.int32)
    s = (((amax + (0x7FFFFF - most)) >> 23) - unit).clamp_min(1)
    y = x.abs() * torch.exp2((127 - unit - s).double()).float().repeat_interleave(GROUP) * 2.0 ** -112
    low = y.view(torch.int32)
    code = (low + ((dither << (shift - 16)) | (1 << (shift - 17))).to(torch.int32)) >> shift
    if bits == 4:
        code = torch.where((low > 0) & (code == 0), torch.ones_like(code), code)
    else:
        code = code | ((x.view(torch.int32) >> 24) & 0x80)
    return code.to(torch.uint8), s.to(torch.uint8)


def _decode(code, scale, bits):
    c = code.to(torch.int32)
    unit = 8 if bits == 3 else 0
    y = ((c & (0x7F if bits == 3 else 0xFF)) << (23 - bits)).view(torch.float32) * 2.0 ** 112
    y = y * torch.exp2((scale.to(torch.int32) - (127 - unit)).double()).float().repeat_interleave(GROUP)
    return torch.where(c >= 128, -y, y) if bits == 3 else y


def _single(x):
    """The binary32 value nearest to x."""
    return float(torch.tensor(x, dtype=torch.float32))


def _adamw(st):
    case = st["case"]
    f = _single
    b1, b2, step = ADAM["beta1"], ADAM["beta2"], st["step"]
    g = functools.reduce(torch.add, [t.float() for t in st["grads"]])
    if case["grads"] > 1:
        g = torch.div(g, torch.full_like(g, case["grads"]))
    if case["bits"] == 32:
        m, v = st["m"], st["v"]
    else:
        m, v = _decode(st["m"], st["m_scale"], 3), _decode(st["v"], st["v_scale"], 4).square()
    m = m * f(b1) + g * f(1.0 - b1)
    v = v * f(b2) + g * g * f(1.0 - b2)
    r = torch.sqrt(v)
    u = torch.div(m, r * f(1.0 / math.sqrt(1.0 - b2 ** step)) + f(ADAM["eps"]))
    keep = 1.0 - torch.tensor(st["decay"], device=DEV) * f(ADAM["lr"])
    theta = st["theta"] * keep.repeat_interleave(st["lengths"]) - u * f(ADAM["lr"] / (1.0 - b1 ** step))
    if case["bits"] == 32:
        st["theta"], st["m"], st["v"] = theta, m, v
        return theta, m, v
    count = torch.arange(len(st["sizes"]), device=DEV)
    start = torch.tensor(st["at"], device=DEV).repeat_interleave(st["lengths"])
    key = _mix((_mix(torch.full_like(count, (0x9E3779B9 * step) & 0xFFFFFFFF)) + 0x9E3779B9 * (count + 1)) & 0xFFFFFFFF)
    h = _mix(((torch.arange(theta.numel(), device=DEV) - start) * 0x9E3779B1 +
              key.repeat_interleave(st["lengths"])) & 0xFFFFFFFF)
    st["theta"] = theta
    st["m"], st["m_scale"] = _encode(m, 3, h & 0xFFFF)
    st["v"], st["v_scale"] = _encode(r, 4, h >> 16)
    return theta, _decode(st["m"], st["m_scale"], 3), _decode(st["v"], st["v_scale"], 4).square()


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "logprobs":
        return tuple(_logprobs(st, case["temp"], case["top"])[0])
    if op == "logprobs_train":
        out, *rest = _logprobs(st, 1.0, 0)
        return tuple(out) + (_logprobs_gradient(st, out[2], *rest),)
    if op == "adamw":
        return _adamw(st)
    x, gain = _by_head(st, "x"), _gains(st)
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    if op == "qk":
        return _unpadded(st, _rotate(st, x * inv * gain, 1.0))
    d = _rotate(st, _by_head(st, "dy"), -1.0)
    xh, gy = x * inv, d * gain
    dx = inv * (gy - xh * (gy * xh).mean(-1, keepdim=True))
    terms = (d * xh * (st["pos"] >= 0)[:, None, None]).sum(0)
    return _unpadded(st, dx), terms[:case["q"]].sum(0), terms[case["q"]:].sum(0)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- work ----

def work(case):
    op = case["op"]
    if op == "logprobs":
        n = case["M"] * case["V"]
        return {"bytes": n * SIZE[case["type"]] + case["M"] * (8 + 12 + 12 * case["top"]), "flops": 20 * n}
    if op == "logprobs_train":
        # the logits in, their gradient out
        n = case["M"] * case["V"]
        return {"bytes": 2 * n * SIZE[case["type"]] + case["M"] * 24, "flops": 40 * n}
    if op.startswith("qk"):
        n = case["rows"] * (case["q"] + case["k"]) * case["dim"]
        table = 8 * (case["rot"] // 2) * min(case["rows"], case["table"])
        if op == "qk":
            return {"bytes": 2 * n * SIZE[case["type"]] + table + 4 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * SIZE[case["type"]] + table + 4 * case["rows"], "flops": 20 * n}
    n = sum(_sizes(case)[0])
    g = case["grads"] * SIZE[case["type"]]
    if case["bits"] == 32:
        return {"bytes": n * (24 + g), "flops": 15 * n}
    # 8-bit moments in and out, and the values they stand for
    return {"bytes": n * (8 + 4 + 8 + g) + 4 * (n // GROUP), "flops": 40 * n}


# ------------------------------------------------------------------ exact ----

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    D = torch.float64
    if op.startswith("logprobs"):
        M, V = case["M"], case["V"]
        temp = case.get("temp", 1.0)
        parts = []
        step = max(1, (1 << 27) // V)
        for r in range(0, M, step):
            z = st["logits"][r:r + step].to(D) / temp
            t = st["targets"][r:r + step]
            lse = torch.logsumexp(z, 1)
            lp = z - lse[:, None]
            p = lp.exp()
            ent = -torch.nansum(p * lp, 1)
            rows = torch.arange(len(t), device=DEV)
            logp = torch.where(t < 0, torch.zeros_like(lse), lp[rows, t.clamp(min=0)])
            got = [logp, lse, ent]
            if op == "logprobs":
                if case["top"]:
                    got.append(lp.topk(case["top"], 1).values)
            else:
                w = st["dlogp"][r:r + step].to(D) * (t >= 0)
                d = -p * w[:, None]
                if st["dentropy"] is not None:
                    d -= st["dentropy"][r:r + step].to(D)[:, None] * torch.nan_to_num(p * (lp + ent[:, None]))
                d[rows, t.clamp(min=0)] += w
                got.append(d)
            parts.append(got)
        out = [torch.cat(v) for v in zip(*parts)]
        # the alternatives' numbers are whole: they are compared with the plain form's
        return tuple(out) + ((None,) if op == "logprobs" and case["top"] else ())
    if op.startswith("qk"):
        rows, dim, pairs = case["rows"], case["dim"], case["rot"] // 2
        live = st["pos"] >= 0
        i = torch.arange(pairs, device=DEV)
        ia, ib = (2 * i, 2 * i + 1) if case["layout"] == "adjacent" else (i, i + pairs)
        at = st["pos"].clamp(min=0).long()
        turn = torch.complex(st["cos"][at].to(D), st["sin"][at].to(D))

        def spin(v, by):
            w = torch.complex(v[..., ia], v[..., ib]) * by[:, None, :]
            v = v.clone()
            v[..., ia], v[..., ib] = w.real, w.imag
            return v

        def whole(q, k):
            y = torch.cat([q.flatten(1), k.flatten(1)], 1)
            return torch.where(live[:, None], y, st["out"].to(D))

        def heads(t):
            t = t.to(D).reshape(rows, -1, dim)
            return t[:, :case["q"]], t[:, case["q"]:]

        def rms(v):
            return (v.square().sum(-1, keepdim=True) / dim + EPS).sqrt()

        pair = list(zip(heads(st["x"]), (st["q_gain"].to(D), st["k_gain"].to(D))))
        if op == "qk":
            return whole(*[spin(v / rms(v) * gain, turn) for v, gain in pair])
        dx, dgain = [], []
        for (v, gain), d in zip(pair, heads(st["dy"])):
            d = spin(d, turn.conj())
            vh = v / rms(v)
            t = d * gain
            dx.append((t - vh * (t * vh).sum(-1, keepdim=True) / dim) / rms(v))
            dgain.append((d * vh)[live].sum((0, 1)))
        return whole(*dx), dgain[0], dgain[1]
    g = sum(t.to(D) for t in st["grads"]) / case["grads"]
    m0, v0 = st["m"], st["v"]
    if case["bits"] == 8:
        c = v0.to(D)
        e = torch.floor(c / 16)
        root = torch.where(e == 0, c / 16 * 2.0 ** -14, (1 + (c - 16 * e) / 16) * torch.exp2(e - 15))
        m0 = m0.view(torch.float8_e4m3fn).to(D) * torch.exp2(st["m_scale"].to(D) - 127).repeat_interleave(GROUP)
        v0 = (root * torch.exp2(st["v_scale"].to(D) - 127).repeat_interleave(GROUP)) ** 2
    b1, b2, n = ADAM["beta1"], ADAM["beta2"], st["step"]
    m = b1 * m0.to(D) + (1 - b1) * g
    v = b2 * v0.to(D) + (1 - b2) * g * g
    keep = 1 - ADAM["lr"] * torch.tensor(st["decay"], dtype=D, device=DEV).repeat_interleave(st["lengths"])
    hat = m / (1 - b1 ** n) / ((v / (1 - b2 ** n)).sqrt() + ADAM["eps"])
    theta = st["theta"].to(D) * keep - ADAM["lr"] * hat
    # which of two neighbouring 8-bit values is kept hangs on the bits before it
    return (theta, None, None) if case["bits"] == 8 else (theta, m, v)
