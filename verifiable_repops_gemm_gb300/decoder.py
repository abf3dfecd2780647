"""One transformer decoder layer, forward and backward, built only from the
library's order-fixed operators: the workload of a verifiable training step on
a Llama-style model ("Verde与RepOps" §4.3, the Llama-1B training measurement),
driven with synthetic weights.

Layer (pre-norm, causal, grouped-query attention):

    h    = RMSNorm(x; g1)
    qkv  = h W_qkv                                  one GEMM
    q, k = rotary(q, k)                             in place, the heads' pairs
                                                    rotated to each token's position
                                                    (qk_norm: each head normed first,
                                                    in the same pass)
    for every sequence (each GEMM call covers every query head; the
    `group` query heads of a key/value head share its K and V):
        S = (Q K^T) / sqrt(d_head)                  batched GEMM, alpha epilogue,
                                                    tiles above the diagonal skipped
        P = causal softmax of every head's rows     one row-operator call
        O = P V                                     batched GEMM over k <= i only,
                                                    written as the heads' column blocks
    x    = x + O W_o                                GEMM, residual epilogue (in place)
    h    = RMSNorm(x; g2)
    SwiGLU MLP (mlp="swiglu", Llama):
        [g | u] = h W_gu                            one GEMM, gate and up side by side
        a    = SiLU(g) * u                          element-wise kernel
        x    = x + a W_down                         GEMM, residual epilogue
    GeLU MLP (mlp="gelu"):
        a    = GeLU(h W_up + b_up)                  GEMM, bias epilogue; GeLU kernel
        x    = x + a W_down + b_down                GEMM, bias + residual epilogue

The causal attention GEMMs run over the band where the probabilities are not
+0 (P V over k <= i; the gradients P^T dO and dS^T Q over k >= i, dS K over
k <= i): the skipped terms would add fl(+0 * v) = +-0 to each chain, so the
bits equal those of the full chains while the work halves.

`backward` runs the layer's backward pass from saved activations: weight,
bias and gain gradients and the input gradient, every step again a library
call (transposed GEMMs, the backward row operators, column sums, the inverse
rotation); the key and value gradients of a key/value head accumulate its
query heads in head order through the GEMM's residual epilogue.

Sandwich blocks (post_norm, gated, residual_scale): each block's output passes
through a norm of its own, a learned gate and a residual scale before the
residual sum -- x = x + s * (gate * RMSNorm(f)) -- and the edge between the two
blocks, with the norm before the MLP, is one call (rmsnorm_residual).

Queries and keys: `qk_norm` norms each head with a gain of its own kind (gq, gk)
before the rotation; `rope_layout`, `rope_dim` and `rope_factor` choose which
columns of a head pair up, how many are rotated, and frequencies for longer
contexts (head_norm_rope, which does all of it in one pass).

8-bit checkpoints: `activations(bits=8)` keeps x, qkv, the attention output
and the MLP's input to its activation as 8-bit rows with a scale for every 128
columns (about a quarter of their bytes), and no norm outputs, activations or
probabilities: `backward` recomputes those from the restored rows.  Its bits are
those of the binary32 backward on the restored activations.

8-bit weights: `quantize_weights` and `forward_i8` run the layer's four weight
products on 8-bit rows (a scale a token) and 8-bit weights (a scale a channel)
for inference (gemm_i8).

Every step is a library call (this module only slices tensors); the bits of
the result depend on nothing but the inputs.  In the GeLU layer, GeLU runs as
its own kernel by default: inside the GEMM's epilogue it measured 2.5x its
stand-alone cost (the GEMM is bound by the FP32 pipe, and its epilogue runs on
few warps), more than the memory pass it saves; `gelu_epilogue=True` fuses it
anyway.  `fused=False` runs every epilogue as a separate step (GEMM, then
element-wise adds in PyTorch): the same bits, more memory traffic; it exists
to measure what the fusion saves.
"""
import math
from dataclasses import dataclass

import torch

from . import (gemm, gemm_batched, gelu, rmsnorm_rows, softmax_rows, ACT_GELU, colsum, gelu_backward,
               rmsnorm_backward, softmax_backward, swiglu, swiglu_backward, rope_frequencies, rope_table, rope,
               rmsnorm_residual, rmsnorm_residual_backward, quantize_rows, dequantize_rows, swiglu_backward_i8,
               rmsnorm_backward_i8, gemm_i8, head_norm_rope, head_norm_rope_backward)

CHECKPOINT_GROUP = 128   # columns that share a scale in an 8-bit checkpoint


@dataclass(frozen=True)
class DecoderConfig:
    d: int = 2048              # model width
    heads: int = 32            # query heads
    kv_heads: int = 8          # key/value heads (grouped-query attention)
    ffn: int = 8192            # MLP width
    seq_len: int = 2048        # tokens per sequence
    eps: float = 1e-5
    mlp: str = "swiglu"        # "swiglu" (Llama: gate and up, no biases) or "gelu" (up + bias)
    rope_base: float = 500000.0  # rotary base; 0 turns the rotary embedding off
    post_norm: bool = False    # a norm after each block (gains p1, p2)
    gated: bool = False        # a learned gate on each block's output (a1, a2)
    residual_scale: float = 1.0  # the scale of a block's output in the residual sum
    qk_norm: bool = False      # a norm of each query and key head before its rotation (gains gq, gk)
    rope_layout: str = "adjacent"  # a rotation's pairs: "adjacent" (2i, 2i + 1) or "halves" (i, i + pairs)
    rope_dim: int = 0          # columns of a head that are rotated, its first ones (0: all)
    rope_factor: float = 1.0   # contexts this many times as long: scaled frequencies
    rope_original: float = 0.0  # the original context's tokens (0: all frequencies scaled alike)

    @property
    def sandwich(self) -> bool:
        return self.post_norm or self.gated or self.residual_scale != 1.0

    @property
    def d_head(self) -> int:
        return self.d // self.heads

    @property
    def qk_width(self) -> int:
        return (self.heads + self.kv_heads) * self.d_head

    @property
    def qkv_width(self) -> int:
        return self.d + 2 * self.kv_heads * self.d_head

    def flops(self, tokens: int) -> float:
        """Multiply-adds x 2 of the layer's GEMMs, attention counted over the
        causal band only (S (S + 1) / 2 scores per head): the work the layer
        needs, not the full score matrix."""
        d, f, w = self.d, self.ffn, self.qkv_width
        seqs = tokens // self.seq_len
        S = self.seq_len
        attn = 2 * 2.0 * seqs * self.heads * (S * (S + 1) / 2) * self.d_head
        mlp = 3 * d * f if self.mlp == "swiglu" else 2 * d * f
        return 2.0 * tokens * (d * w + d * d + mlp) + attn


def weight_shapes(cfg: DecoderConfig) -> dict:
    """Every weight of a layer and its shape, in a fixed order."""
    d, w, f = cfg.d, cfg.qkv_width, cfg.ffn
    if cfg.mlp == "swiglu":
        out = {"g1": (d,), "w_qkv": (d, w), "w_o": (d, d), "g2": (d,), "w_gu": (d, 2 * f), "w_down": (f, d)}
    elif cfg.mlp == "gelu":
        out = {"g1": (d,), "w_qkv": (d, w), "w_o": (d, d), "g2": (d,), "w_up": (d, f), "b_up": (f,),
               "w_down": (f, d), "b_down": (d,)}
    else:
        raise ValueError("mlp must be 'swiglu' or 'gelu'")
    if cfg.post_norm:
        out.update(p1=(d,), p2=(d,))
    if cfg.gated:
        out.update(a1=(d,), a2=(d,))
    if cfg.qk_norm:
        out.update(gq=(cfg.d_head,), gk=(cfg.d_head,))
    return out


GAINS = ("g1", "g2", "p1", "p2", "a1", "a2", "gq", "gk")


def init_weights(cfg: DecoderConfig, seed: int, device) -> dict:
    """Synthetic weights: N(0, 0.02) matrices and biases, norm gains and gates
    N(1, 0.1); seeded, generated on `device`."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    out = {}
    for name, shape in weight_shapes(cfg).items():
        t = torch.randn(shape, generator=g, device=device, dtype=torch.float32)
        out[name] = t * 0.1 + 1.0 if name in GAINS else t * 0.02
    return out


def rope_tables(cfg: DecoderConfig, device):
    """(cos, sin), seq_len x pairs, of the layer's rotary embedding, or None when
    it is off: pairs = rope_dim/2 (d_head/2), frequencies base^(-i/pairs) from the
    binary32 value of ln(base), scaled where rope_factor asks for it, angles
    p * f_i for positions p < seq_len."""
    if not cfg.rope_base:
        return None
    if cfg.rope_dim % 2 or not 0 <= cfg.rope_dim <= cfg.d_head:
        raise ValueError("rope_dim must be even and at most a head's width")
    freq = rope_frequencies((cfg.rope_dim or cfg.d_head) // 2, math.log(cfg.rope_base), device,
                            factor=cfg.rope_factor, original=cfg.rope_original)
    return rope_table(cfg.seq_len, freq)


def _turn(cfg: DecoderConfig, tables):
    """head_norm_rope's keyword arguments for the layer's rotation."""
    cos, sin = tables if tables is not None else (None, None)
    return dict(cos=cos, sin=sin, layout=cfg.rope_layout, period=cfg.seq_len)


def _rotate(qkv, w: dict, cfg: DecoderConfig, tables):
    """The norms (qk_norm) and the rotary embedding of the query and key heads,
    in place: columns [0, (heads + kv_heads) * d_head) of every row, position =
    the row's index within its sequence."""
    if cfg.qk_norm or cfg.rope_layout != "adjacent" or cfg.rope_dim:
        qk = qkv[:, :cfg.qk_width]
        gains = dict(q_gain=w["gq"], k_gain=w["gk"], eps=cfg.eps) if cfg.qk_norm else {}
        head_norm_rope(qk, cfg.heads, cfg.kv_heads, out=qk, **gains, **_turn(cfg, tables))
    elif tables is not None:
        rope(qkv, cfg.heads + cfg.kv_heads, tables[0], tables[1], first=0, period=cfg.seq_len)


def _rotate_backward(dqkv, qk, w: dict, cfg: DecoderConfig, tables, g: dict, o: dict):
    """_rotate's backward in place on dqkv; with qk_norm from the heads before
    their norms (qk), the gains' gradients into g."""
    if cfg.qk_norm:
        d = dqkv[:, :cfg.qk_width]
        _, g["gq"], g["gk"] = head_norm_rope_backward(d, qk, cfg.heads, cfg.kv_heads, q_gain=w["gq"], k_gain=w["gk"],
                                                      eps=cfg.eps, dx=d, dq_gain=o.get("gq"), dk_gain=o.get("gk"),
                                                      **_turn(cfg, tables))
    elif cfg.rope_layout != "adjacent" or cfg.rope_dim:
        d = dqkv[:, :cfg.qk_width]
        head_norm_rope(d, cfg.heads, cfg.kv_heads, out=d, inverse=True, **_turn(cfg, tables))
    elif tables is not None:
        rope(dqkv, cfg.heads + cfg.kv_heads, tables[0], tables[1], first=0, period=cfg.seq_len, inverse=True)


def _after(stream, *others):
    """Work queued on `stream` from now on waits for everything queued so far
    on `others`."""
    for o in others:
        e = torch.cuda.Event()
        e.record(o)
        stream.wait_event(e)


def side_streams(cfg: DecoderConfig, tokens: int, device):
    """The side streams one layer's attention runs its independent work on:
    three per sequence (the scores, softmax and products of a sequence, or in
    the backward its dP / dQ; the dV chain; the dK chain)."""
    return [torch.cuda.Stream(device) for _ in range(tokens // cfg.seq_len * 3)]


def _per_kv(t, rows, col0, kv, group, h, dh):
    """(kv, S, dh) view of query head h of every key/value group: the column
    block (k*group + h)*dh of rows, k = 0 .. kv-1 (a batch stride of
    group*dh)."""
    return t[rows, col0:col0 + kv * group * dh].unflatten(1, (kv, group, dh))[:, :, h, :].transpose(0, 1)


def _kv(t, rows, col0, kv, dh):
    """(kv, S, dh) view of the key or value heads: column block col0 + k*dh."""
    return t[rows, col0:col0 + kv * dh].unflatten(1, (kv, dh)).transpose(0, 1)


def _heads(t, rows, col0, n, dh):
    """(n, S, dh) view of n consecutive heads: column block col0 + h*dh."""
    return t[rows, col0:col0 + n * dh].unflatten(1, (n, dh)).transpose(0, 1)


def attention(qkv, cfg: DecoderConfig, out, scores, probs=None, streams=None, fused: bool = False):
    """Causal grouped-query attention of every sequence into `out` (T x d).
    scores: (sequences * kv_heads, group, S, S) scratch (or (kv_heads, group,
    S, S), shared by the sequences in turn); probs: optional buffer shaped
    like the first that keeps every head's softmax output for the backward
    pass.

    fused: one launch of the fused kernel (repops_attention_causal_f32:
    scores, causal softmax and the banded product per block of 16 query rows in
    shared memory) where its limits allow; it computes the same bits as the
    operators below and needs no S x S scratch (`scores` is not touched), but
    it is slower at decoder sizes, so the unfused operators are the default.
    Unfused: one GEMM call covers every query head of a sequence: a key/value
    head's K or V is shared by the `group` consecutive query heads of its
    group.  streams (from
    `side_streams`): the sequences run concurrently -- their outputs are
    disjoint, so the bits do not change -- and the caller's stream waits for
    all of them."""
    S, dh, kv, H = cfg.seq_len, cfg.d_head, cfg.kv_heads, cfg.heads
    k0, v0 = cfg.d, cfg.d + kv * dh
    scale = 1.0 / float(dh) ** 0.5
    seqs = qkv.shape[0] // S
    if fused:
        from . import attention_causal
        from ._capi import RepopsError, ERR_UNSUPPORTED
        try:
            attention_causal(qkv[:, :H * dh], qkv[:, k0:k0 + kv * dh], qkv[:, v0:v0 + kv * dh], out,
                             seq_len=S, heads=H, kv_heads=kv, scale=scale,
                             probs=probs.view(seqs * H, S, S) if probs is not None else None)
            return
        except RepopsError as e:
            if e.code != ERR_UNSUPPORTED:
                raise
    buf = probs if probs is not None else scores
    shared = buf.shape[0] < seqs * kv
    main = torch.cuda.current_stream()
    prev, joined = None, []
    if streams is not None:
        fork = torch.cuda.Event()
        fork.record(main)
    for s in range(seqs):
        rows = slice(s * S, (s + 1) * S)
        sc = (buf if shared else buf[s * kv:(s + 1) * kv]).view(H, S, S)       # head q = k*group + h
        st = main if streams is None else streams[3 * s]
        if streams is not None:
            st.wait_event(fork)
            if shared and prev is not None:    # a shared scratch is reused after the previous sequence
                _after(st, prev)
        with torch.cuda.stream(st):
            # tiles wholly above the diagonal are skipped: the causal softmax
            # never reads them
            gemm_batched(_heads(qkv, rows, 0, H, dh), _kv(qkv, rows, k0, kv, dh).transpose(1, 2), out=sc,
                         alpha=scale, causal_first=0)
            P = sc.view(H * S, S)
            softmax_rows(P, out=P, causal_first=0, causal_period=S)
            # P is +0 past the diagonal: row i's chain stops at k = i
            gemm_batched(sc, _kv(qkv, rows, v0, kv, dh), out=_heads(out, rows, 0, H, dh), k_hi=0)
        prev = st
        joined.append(st)
    if streams is not None:
        _after(main, *joined)


def forward(x, w: dict, cfg: DecoderConfig, *, fused: bool = True, gelu_epilogue: bool = False,
            work: dict = None, save: dict = None, fused_attention: bool = False):
    """Runs the layer on x (T x d, T a multiple of seq_len) in place and
    returns it.  `work`: reusable buffers from `workspace` (allocated when
    absent).  `fused`: biases and residual sums in the products' epilogues, a
    sandwich layer's edges in one call; without it they are steps of their own.
    `gelu_epilogue`: GeLU in the product's epilogue too.  `save`: a dict (from
    `activations`) that receives what `backward` needs; a GeLU layer's MLP then
    keeps its GeLU input and runs GeLU as its own kernel, whatever these two
    say.  The bits are the same each way."""
    T = x.shape[0]
    if T % cfg.seq_len:
        raise ValueError("tokens must be a whole number of sequences")
    ws = work if work is not None else workspace(cfg, T, x.device)
    f = cfg.ffn
    if save is not None and save.get("bits") == 8:
        return _forward_checkpointed(x, w, cfg, ws, save, fused, fused_attention)
    if save is not None:
        save["x0"].copy_(x)
        h, qkv, attn, a = save["h1"], save["qkv"], save["attn"], save["a"]
    else:
        h, qkv, attn, a = ws["h"], ws["qkv"], ws["attn"], ws["a"]
    rmsnorm_rows(x, w["g1"], cfg.eps, out=h)
    gemm(h, w["w_qkv"], out=qkv)
    if cfg.qk_norm and save is not None:
        save["qk"].copy_(qkv[:, :cfg.qk_width])
    _rotate(qkv, w, cfg, ws["rope"])
    attention(qkv, cfg, attn, ws["scores"], save["probs"] if save is not None else None, ws.get("streams"),
              fused=fused_attention)
    if cfg.sandwich:
        f1 = gemm(attn, w["w_o"], out=save["f1"] if save is not None else ws["tmp_d"])
        h = save["h2"] if save is not None else h
        steps = None if fused else ws["tmp_d"]
        _edge(x, f1, w, cfg, 1, h, steps)
        if save is not None:
            save["x1"].copy_(x)
        f2 = _mlp(h, w, cfg, ws, save, save["f2"] if save is not None else ws["tmp_d"], fused, gelu_epilogue)
        _edge(x, f2, w, cfg, 2, steps=steps)
        return x
    if fused:
        gemm_batched(attn, w["w_o"], out=x, residual=x)
    else:
        x += gemm(attn, w["w_o"], out=ws["tmp_d"])
    if save is not None:
        save["x1"].copy_(x)
        h = save["h2"]
    rmsnorm_rows(x, w["g2"], cfg.eps, out=h)
    if cfg.mlp == "swiglu":
        gu = save["gu"] if save is not None else ws["gu"]
        gemm(h, w["w_gu"], out=gu)
        swiglu(gu[:, :f], gu[:, f:], out=a)
        if fused:
            gemm_batched(a, w["w_down"], out=x, residual=x)
        else:
            x += gemm(a, w["w_down"], out=ws["tmp_d"])
        return x
    if save is not None:
        gemm_batched(h, w["w_up"], out=save["pre"], bias=w["b_up"])
        gelu(save["pre"], out=a)
        gemm_batched(a, w["w_down"], out=x, bias=w["b_down"], residual=x)
    elif fused:
        if gelu_epilogue:
            gemm_batched(h, w["w_up"], out=a, bias=w["b_up"], act=ACT_GELU)
        else:
            gemm_batched(h, w["w_up"], out=a, bias=w["b_up"])
            gelu(a, out=a)
        gemm_batched(a, w["w_down"], out=x, bias=w["b_down"], residual=x)
    else:
        gemm(h, w["w_up"], out=a)
        a += w["b_up"]
        gelu(a, out=a)
        y = gemm(a, w["w_down"], out=ws["tmp_d"])
        y += w["b_down"]
        x += y
    return x


def _edge(x, f, w, cfg: DecoderConfig, k: int, h=None, steps=None):
    """The edge after block k (1 attention, 2 MLP) in place on x; with h, the
    norm before the MLP into it.  steps: scratch like x (f's own memory is fine)
    to take the edge in as operators of their own."""
    post, gate = w.get("p%d" % k), w.get("a%d" % k)
    if steps is None:
        rmsnorm_residual(x, f, w["g2"] if h is not None else None, cfg.eps, post_gain=post, gate=gate,
                         alpha=cfg.residual_scale, y=x, h=h)
        return
    t = f if post is None else rmsnorm_rows(f, post, cfg.eps, out=steps)
    t = t if gate is None else torch.mul(t, gate, out=steps)
    x += torch.mul(t, cfg.residual_scale, out=steps)
    if h is not None:
        rmsnorm_rows(x, w["g2"], cfg.eps, out=h)


def _mlp(h, w, cfg: DecoderConfig, ws, save, out, fused: bool = True, gelu_epilogue: bool = False):
    """The MLP of h (without the residual) into `out`, its activations where
    `save` keeps them (in 8 bits only GeLU's input, which GeLU then replaces)."""
    f = cfg.ffn
    kept8 = save is not None and save.get("bits") == 8
    keep = ws if save is None or kept8 else save
    a = keep["a"]
    if cfg.mlp == "swiglu":
        gu = keep["gu"]
        gemm(h, w["w_gu"], out=gu)
        swiglu(gu[:, :f], gu[:, f:], out=a)
        return gemm(a, w["w_down"], out=out)
    if save is None and not fused:
        gemm(h, w["w_up"], out=a)
        a += w["b_up"]
        y = gemm(gelu(a, out=a), w["w_down"], out=out)
        y += w["b_down"]
        return y
    if save is None and gelu_epilogue:
        gemm_batched(h, w["w_up"], out=a, bias=w["b_up"], act=ACT_GELU)
        return gemm_batched(a, w["w_down"], out=out, bias=w["b_down"])
    pre = a if keep is ws else save["pre"]
    gemm_batched(h, w["w_up"], out=pre, bias=w["b_up"])
    if kept8:
        _keep(save, "pre", pre)
    gelu(pre, out=a)
    return gemm_batched(a, w["w_down"], out=out, bias=w["b_down"])


def _keep(save, name, t):
    """t's rows in 8 bits into the checkpoint `name`."""
    q, s = save[name]
    quantize_rows(t, group=CHECKPOINT_GROUP, out=q, scale=s)


def _restore(save, name, out):
    q, s = save[name]
    return dequantize_rows(q, s, group=CHECKPOINT_GROUP, out=out)


def _forward_checkpointed(x, w, cfg: DecoderConfig, ws, save, fused, fused_attention):
    """forward(save=...) for activations(bits=8): the same x, the activations
    quantised as they are made."""
    h, qkv, attn, tmp = ws["h"], ws["qkv"], ws["attn"], ws["tmp_d"]
    _keep(save, "x0", x)
    rmsnorm_rows(x, w["g1"], cfg.eps, out=h)
    gemm(h, w["w_qkv"], out=qkv)
    if cfg.qk_norm:                          # the heads' norms are computed again from what they normed
        _keep(save, "qkv", qkv)
    _rotate(qkv, w, cfg, ws["rope"])
    if not cfg.qk_norm:
        _keep(save, "qkv", qkv)
    attention(qkv, cfg, attn, ws["scores"], None, ws.get("streams"), fused=fused_attention)
    _keep(save, "attn", attn)
    if cfg.sandwich:
        f1 = gemm(attn, w["w_o"], out=tmp)
        _keep(save, "f1", f1)
        _edge(x, f1, w, cfg, 1, h, None if fused else tmp)
    else:
        if fused:
            gemm_batched(attn, w["w_o"], out=x, residual=x)
        else:
            x += gemm(attn, w["w_o"], out=tmp)
        rmsnorm_rows(x, w["g2"], cfg.eps, out=h)
    _keep(save, "x1", x)
    if cfg.sandwich:
        f2 = _mlp(h, w, cfg, ws, save, tmp)
        _keep(save, "f2", f2)
        _edge(x, f2, w, cfg, 2, steps=None if fused else tmp)
    elif cfg.mlp == "swiglu":
        gemm(h, w["w_gu"], out=ws["gu"])
        swiglu(ws["gu"][:, :cfg.ffn], ws["gu"][:, cfg.ffn:], out=ws["a"])
        if fused:
            gemm_batched(ws["a"], w["w_down"], out=x, residual=x)
        else:
            x += gemm(ws["a"], w["w_down"], out=tmp)
    else:
        gemm_batched(h, w["w_up"], out=ws["a"], bias=w["b_up"])
        _keep(save, "pre", ws["a"])
        gelu(ws["a"], out=ws["a"])
        gemm_batched(ws["a"], w["w_down"], out=x, bias=w["b_down"], residual=x)
    if cfg.mlp == "swiglu":
        _keep(save, "g", ws["gu"][:, :cfg.ffn])
        _keep(save, "u", ws["gu"][:, cfg.ffn:])
    return x


WEIGHT_MATRICES = ("w_qkv", "w_o", "w_gu", "w_up", "w_down")


def quantize_weights(w: dict, cfg: DecoderConfig) -> dict:
    """The layer's weight matrices in 8 bits for `forward_i8`: name -> (whole
    numbers (N, K), a row for each output channel; scales (N,))."""
    out = {}
    for name in WEIGHT_MATRICES:
        if name in w:
            q, s = quantize_rows(w[name].t().contiguous())
            out[name] = (q, s.view(-1))
    return out


def forward_i8(x, w: dict, w8: dict, cfg: DecoderConfig, *, work: dict = None, fused_attention: bool = False):
    """The layer on x in place with 8-bit weight products (inference): every
    operand row is quantised with a scale of its own just before its product
    (quantize_rows, gemm_i8 with `quantize_weights`' w8); norms, rotary
    embedding, attention and residual sums stay binary32."""
    T, f = x.shape[0], cfg.ffn
    if T % cfg.seq_len:
        raise ValueError("tokens must be a whole number of sequences")
    ws = work if work is not None else workspace(cfg, T, x.device)

    def product(rows, name, out, bias=None):
        q, s = quantize_rows(rows)
        wq, wscale = w8[name]
        return gemm_i8(q, wq.t(), s.view(-1), wscale, out=out, bias=bias)

    h = rmsnorm_rows(x, w["g1"], cfg.eps, out=ws["h"])
    qkv = product(h, "w_qkv", ws["qkv"])
    _rotate(qkv, w, cfg, ws["rope"])
    attention(qkv, cfg, ws["attn"], ws["scores"], None, ws.get("streams"), fused=fused_attention)
    _edge(x, product(ws["attn"], "w_o", ws["tmp_d"]), w, cfg, 1, h)
    if cfg.mlp == "swiglu":
        gu = product(h, "w_gu", ws["gu"])
        a = swiglu(gu[:, :f], gu[:, f:], out=ws["a"])
        f2 = product(a, "w_down", ws["tmp_d"])
    else:
        a = product(h, "w_up", ws["a"], bias=w["b_up"])
        f2 = product(gelu(a, out=a), "w_down", ws["tmp_d"], bias=w["b_down"])
    _edge(x, f2, w, cfg, 2)
    return x


def activations(cfg: DecoderConfig, tokens: int, device, bits: int = 32) -> dict:
    """Buffers for the activations `forward(save=...)` keeps for `backward`
    (every head's attention probabilities included: seqs * heads * S^2).
    bits=8: 8-bit checkpoints instead, (whole numbers, scales) a tensor, of
    what backward does not recompute."""
    e = dict(dtype=torch.float32, device=device)
    group, S = cfg.heads // cfg.kv_heads, cfg.seq_len
    if bits == 8:
        def rows(cols):
            return (torch.empty(tokens, cols, dtype=torch.int8, device=device),
                    torch.empty(tokens, -(-cols // CHECKPOINT_GROUP), **e))

        out = {"bits": 8, "x0": rows(cfg.d), "qkv": rows(cfg.qkv_width), "attn": rows(cfg.d), "x1": rows(cfg.d)}
        if cfg.mlp == "swiglu":
            out.update(g=rows(cfg.ffn), u=rows(cfg.ffn))
        else:
            out["pre"] = rows(cfg.ffn)
        if cfg.sandwich:
            out.update(f1=rows(cfg.d), f2=rows(cfg.d))
        return out
    if bits != 32:
        raise ValueError("bits must be 32 or 8")
    out = {"x0": torch.empty(tokens, cfg.d, **e), "h1": torch.empty(tokens, cfg.d, **e),
           "qkv": torch.empty(tokens, cfg.qkv_width, **e), "attn": torch.empty(tokens, cfg.d, **e),
           "probs": torch.empty(tokens // S * cfg.kv_heads, group, S, S, **e),
           "x1": torch.empty(tokens, cfg.d, **e), "h2": torch.empty(tokens, cfg.d, **e),
           "a": torch.empty(tokens, cfg.ffn, **e)}
    if cfg.mlp == "swiglu":
        out["gu"] = torch.empty(tokens, 2 * cfg.ffn, **e)
    else:
        out["pre"] = torch.empty(tokens, cfg.ffn, **e)
    if cfg.sandwich:
        out.update(f1=torch.empty(tokens, cfg.d, **e), f2=torch.empty(tokens, cfg.d, **e))
    if cfg.qk_norm:
        out["qk"] = torch.empty(tokens, cfg.qk_width, **e)
    return out


def backward(dy, w: dict, cfg: DecoderConfig, saved: dict, *, work: dict = None, grads: dict = None):
    """Gradients of the layer given dy = dL/d(output): returns (dx, grads) with
    grads holding one tensor per weight of `init_weights` (written into the
    tensors of `grads` when given, e.g. views of one flat gradient buffer).
    dy is consumed (used as scratch) and dx is returned in its storage; a
    SwiGLU layer's saved["gu"] is overwritten with its gradient.  Every step
    is a library call:

        SwiGLU MLP:
          dW_down = a^T dy, da = dy W_down^T
          [dg | du] = SwiGLU'(g, u; da), dW_gu = h2^T [dg | du], dh2 = [dg | du] W_gu^T
        GeLU MLP:
          dW_down = a^T dy, db_down = colsum(dy), da = dy W_down^T
          dpre = GeLU'(pre) da, dW_up = h2^T dpre, db_up = colsum(dpre), dh2 = dpre W_up^T
        dx1 = RMSNorm'(x1; dh2) + dy, dg2 = colsum(dh2 * xhat2)
        dW_o = attn^T dx1, dattn = dx1 W_o^T
        attention, per sequence and key/value head k (its query heads h):
            dP_h = dO_h V_k^T (on and below the diagonal);
            dV_k = sum_h P_h^T dO_h (head order, k >= i)
            dS_h = causal softmax'(P_h; dP_h)
            dQ_h = s dS_h K_k (k <= i);  dK_k = sum_h s dS_h^T Q_h (head order,
            k >= i), s = 1/sqrt(d_head)
        dq, dk rotated back (the rotary embedding's transpose; with qk_norm the
        heads' norms too, and dgq, dgk)
        dW_qkv = h1^T dqkv, dh1 = dqkv W_qkv^T
        dx0 = RMSNorm'(x0; dh1) + dx1, dg1 = colsum(dh1 * xhat1)

    In a sandwich layer the edges' backward (rmsnorm_residual_backward) stands
    before the MLP's and in the place of RMSNorm'(x1; dh2) + dy: it splits dy
    into the residual's gradient and the block's, and gives dp2, da2 and dg2, dp1,
    da1.  From 8-bit checkpoints the norms' and SwiGLU's backward read the kept
    rows and write the norm outputs and activations the weight gradients need.
    """
    T, f = dy.shape[0], cfg.ffn
    kept8 = saved.get("bits") == 8
    ws = work if work is not None else backward_workspace(cfg, T, dy.device, bits=8 if kept8 else 32)
    if kept8 and "h" not in ws:
        raise ValueError("a backward pass from 8-bit checkpoints needs scratch of backward_workspace(bits=8)")
    g = {}
    o = grads if grads is not None else {}
    dm = dy                                  # the MLP's gradient
    if cfg.sandwich:
        f2 = _restore(saved, "f2", ws["t_f"]) if kept8 else saved["f2"]
        dy, dm = _edge_backward(dy, None, None, f2, w, cfg, 2, g, o, ws["t_e"])
    if kept8:
        dgu, dh2, a = _mlp_backward_i8(dm, w, cfg, saved, ws, g, o)
    else:
        a = saved["a"]
        g["w_down"] = gemm(a.t(), dm, out=o.get("w_down"))
        da = gemm(dm, w["w_down"].t(), out=ws["t_ffn"])
        if cfg.mlp == "swiglu":
            gu = saved["gu"]
            swiglu_backward(gu[:, :f], gu[:, f:], da, dg=gu[:, :f], du=gu[:, f:])     # gu <- [dg | du]
            g["w_gu"] = gemm(saved["h2"].t(), gu, out=o.get("w_gu"))
            dh2 = gemm(gu, w["w_gu"].t(), out=ws["t_d"])
        else:
            g["b_down"] = colsum(dm, out=o.get("b_down"))
            dpre = gelu_backward(saved["pre"], da, out=da)
            g["w_up"] = gemm(saved["h2"].t(), dpre, out=o.get("w_up"))
            g["b_up"] = colsum(dpre, out=o.get("b_up"))
            dh2 = gemm(dpre, w["w_up"].t(), out=ws["t_d"])
    dblock = None
    if cfg.sandwich:
        f1 = _restore(saved, "f1", ws["t_f"]) if kept8 else saved["f1"]
        x1 = _restore(saved, "x1", ws["h"]) if kept8 else saved["x1"]
        dx1, dblock = _edge_backward(dy, dh2, x1, f1, w, cfg, 1, g, o, ws["t_e"])
        if kept8:
            rmsnorm_rows(x1, w["g2"], cfg.eps, out=ws["h"])
    elif kept8:
        q, s = saved["x1"]
        dx1, g["g2"] = rmsnorm_backward_i8(q, s, w["g2"], cfg.eps, dh2, dx=dy, dgamma=o.get("g2"),
                                           group=CHECKPOINT_GROUP, res=dy, h=ws["h"])
    else:
        dx1, p2 = rmsnorm_backward(saved["x1"], w["g2"], cfg.eps, dh2, dx=dy, dyxh=ws["t_d2"], res=dy)
        g["g2"] = colsum(p2, out=o.get("g2"))
    if dblock is None:
        dblock = dx1
    if kept8:
        g["w_gu" if cfg.mlp == "swiglu" else "w_up"] = gemm(ws["h"].t(), dgu,
                                                            out=o.get("w_gu" if cfg.mlp == "swiglu" else "w_up"))
        attn = _restore(saved, "attn", ws["attn"])
        saved = _recomputed_attention(saved, w, cfg, ws)
    else:
        attn = saved["attn"]
    g["w_o"] = gemm(attn.t(), dblock, out=o.get("w_o"))
    dattn = gemm(dblock, w["w_o"].t(), out=ws["t_d"])
    _attention_backward(dattn, ws["dqkv"], saved, cfg, ws["dp"], ws.get("streams"))
    dqkv = ws["dqkv"]
    _rotate_backward(dqkv, saved.get("qk"), w, cfg, ws["rope"], g, o)
    if kept8:
        dh1 = gemm(dqkv, w["w_qkv"].t(), out=ws["t_d"])
        q, s = saved["x0"]
        dx0, g["g1"] = rmsnorm_backward_i8(q, s, w["g1"], cfg.eps, dh1, dx=dx1, dgamma=o.get("g1"),
                                           group=CHECKPOINT_GROUP, res=dx1, h=ws["h"])
        g["w_qkv"] = gemm(ws["h"].t(), dqkv, out=o.get("w_qkv"))
        return dx0, g
    g["w_qkv"] = gemm(saved["h1"].t(), dqkv, out=o.get("w_qkv"))
    dh1 = gemm(dqkv, w["w_qkv"].t(), out=ws["t_d"])
    dx0, p1 = rmsnorm_backward(saved["x0"], w["g1"], cfg.eps, dh1, dx=dx1, dyxh=ws["t_d2"], res=dx1)
    g["g1"] = colsum(p1, out=o.get("g1"))
    return dx0, g


def _edge_backward(dy, dh, y, f, w, cfg: DecoderConfig, k: int, g: dict, o: dict, df):
    """(dx in dy's storage, the block's gradient in df) of the edge after block
    k; its parameters' gradients into g."""
    post, gate = w.get("p%d" % k), w.get("a%d" % k)
    pre = w["g2"] if dh is not None else None
    dx, df, dpre, dpost, dgate = rmsnorm_residual_backward(
        dy, dh, y, f, pre, cfg.eps, post_gain=post, gate=gate, alpha=cfg.residual_scale, dx=dy, df=df,
        dpre=o.get("g2") if pre is not None else None, dpost=o.get("p%d" % k), dgate=o.get("a%d" % k))
    for name, t in (("g2", dpre), ("p%d" % k, dpost), ("a%d" % k, dgate)):
        if t is not None:
            g[name] = t
    return dx, df


def _mlp_backward_i8(dm, w, cfg: DecoderConfig, saved, ws, g: dict, o: dict):
    """(the gradient of the MLP's first product's output, dh2, the activation) of
    an MLP kept in 8 bits; w_down's (and the biases') gradients into g."""
    f = cfg.ffn
    da = gemm(dm, w["w_down"].t(), out=ws["t_ffn"])
    a = ws["a"]
    if cfg.mlp == "swiglu":
        gu = ws["gu"]
        (gq, gs), (uq, us) = saved["g"], saved["u"]
        swiglu_backward_i8(gq, gs, uq, us, da, dg=gu[:, :f], du=gu[:, f:], group=CHECKPOINT_GROUP, h=a)
        g["w_down"] = gemm(a.t(), dm, out=o.get("w_down"))
        return gu, gemm(gu, w["w_gu"].t(), out=ws["t_d"]), a
    pre = _restore(saved, "pre", ws["pre"])
    gelu(pre, out=a)
    g["w_down"] = gemm(a.t(), dm, out=o.get("w_down"))
    g["b_down"] = colsum(dm, out=o.get("b_down"))
    dpre = gelu_backward(pre, da, out=da)
    g["b_up"] = colsum(dpre, out=o.get("b_up"))
    return dpre, gemm(dpre, w["w_up"].t(), out=ws["t_d"]), a


def _recomputed_attention(saved, w: dict, cfg: DecoderConfig, ws):
    """saved with qkv restored (its heads normed and rotated again where they were
    kept before their norms) and every head's probabilities computed again from it
    (the forward's product and causal softmax)."""
    S, dh, kv, H = cfg.seq_len, cfg.d_head, cfg.kv_heads, cfg.heads
    qkv = _restore(saved, "qkv", ws["qkv"])
    if cfg.qk_norm:
        ws["qk"].copy_(qkv[:, :cfg.qk_width])
        _rotate(qkv, w, cfg, ws["rope"])
    for s in range(qkv.shape[0] // S):
        rows = slice(s * S, (s + 1) * S)
        sc = ws["probs"][s * kv:(s + 1) * kv].view(H, S, S)
        gemm_batched(_heads(qkv, rows, 0, H, dh), _kv(qkv, rows, cfg.d, kv, dh).transpose(1, 2), out=sc,
                     alpha=1.0 / float(dh) ** 0.5, causal_first=0)
        P = sc.view(H * S, S)
        softmax_rows(P, out=P, causal_first=0, causal_period=S)
    return dict(saved, qkv=qkv, probs=ws["probs"], qk=ws.get("qk"))


def _attention_backward(dattn, dqkv, saved, cfg: DecoderConfig, dp, streams):
    """The attention's part of dqkv (before the inverse rotation), per
    sequence, every query head q = k*group + h of key/value head k:
        dP_q = dO_q V_k^T (on and below the diagonal); dV_k = sum_h P_q^T dO_q
        dS_q = causal softmax'(P_q; dP_q)
        dQ_q = s dS_q K_k;  dK_k = sum_h s dS_q^T Q_q
    with dP and dQ one GEMM call per sequence, the dV and dK sums in head
    order through the residual epilogue.  dp: (sequences * kv_heads, group,
    S, S) scratch, or (kv_heads, group, S, S) shared by the sequences in turn.
    With `streams` the sequences run concurrently, and within one the dV
    chain and the dK chain beside dP / dQ; the bits do not change."""
    S, dh, kv, H = cfg.seq_len, cfg.d_head, cfg.kv_heads, cfg.heads
    group = H // kv
    scale = 1.0 / float(dh) ** 0.5
    k0, v0 = cfg.d, cfg.d + kv * dh
    qkv = saved["qkv"]
    seqs = qkv.shape[0] // S
    shared = dp.shape[0] < seqs * kv
    main = torch.cuda.current_stream()
    used, joined = [], []
    if streams is not None:
        fork = torch.cuda.Event()
        fork.record(main)
    for s in range(seqs):
        rows = slice(s * S, (s + 1) * S)
        P = saved["probs"][s * kv:(s + 1) * kv]                               # (kv, group, S, S)
        dP = dp if shared else dp[s * kv:(s + 1) * kv]
        V, K = _kv(qkv, rows, v0, kv, dh), _kv(qkv, rows, k0, kv, dh)
        dV, dK = _kv(dqkv, rows, v0, kv, dh), _kv(dqkv, rows, k0, kv, dh)
        if streams is None:
            sp = sv = sk = main
        else:
            sp, sv, sk = streams[3 * s:3 * s + 3]
            for st in (sp, sv):
                st.wait_event(fork)
            if shared:
                _after(sp, *used)
        with torch.cuda.stream(sp):
            # dP = dO V^T on and below the diagonal (the causal backward reads no more)
            gemm_batched(_heads(dattn, rows, 0, H, dh), V.transpose(1, 2), out=dP.view(H, S, S), causal_first=0)
        with torch.cuda.stream(sv):
            for h in range(group):
                # dV = sum over the group's heads, in head order, of P_h^T dO_h;
                # row i of P^T is +0 before k = i
                gemm_batched(P[:, h].transpose(1, 2), _per_kv(dattn, rows, 0, kv, group, h, dh), out=dV,
                             residual=dV if h else None, k_lo=0)
        with torch.cuda.stream(sp):
            dS = dP.view(H * S, S)
            softmax_backward(P.view(H * S, S), dS, out=dS, causal_first=0, causal_period=S)
            gemm_batched(dP.view(H, S, S), K, out=_heads(dqkv, rows, 0, H, dh), alpha=scale, k_hi=0)
        if streams is not None:
            _after(sk, sp)
        with torch.cuda.stream(sk):
            for h in range(group):
                # dK = sum over the group's heads, in head order, of s dS_h^T Q_h
                gemm_batched(dP[:, h].transpose(1, 2), _per_kv(qkv, rows, 0, kv, group, h, dh), out=dK,
                             alpha=scale, residual=dK if h else None, k_lo=0)
        if streams is not None:
            used = [sp, sv, sk]
            joined += used
    if streams is not None:
        _after(main, *joined)


def backward_workspace(cfg: DecoderConfig, tokens: int, device, bits: int = 32) -> dict:
    """Scratch of `backward`; bits=8 adds what it restores and recomputes from
    8-bit checkpoints (one layer's, reused by every layer)."""
    e = dict(dtype=torch.float32, device=device)
    group, S = cfg.heads // cfg.kv_heads, cfg.seq_len
    seqs = tokens // S
    t_d2 = torch.empty(tokens, cfg.d, **e)
    out = {"t_ffn": torch.empty(tokens, cfg.ffn, **e), "t_d": torch.empty(tokens, cfg.d, **e), "t_d2": t_d2,
           "dqkv": torch.empty(tokens, cfg.qkv_width, **e),
           "dp": torch.empty(seqs * cfg.kv_heads, group, S, S, **e), "rope": rope_tables(cfg, device),
           "streams": side_streams(cfg, tokens, device)}
    if cfg.sandwich:
        out["t_e"] = torch.empty(tokens, cfg.d, **e)
    if bits == 8:
        # h in t_d2's memory, which only the binary32 norms' backward uses
        out.update(h=t_d2, a=torch.empty(tokens, cfg.ffn, **e),
                   qkv=torch.empty(tokens, cfg.qkv_width, **e), attn=torch.empty(tokens, cfg.d, **e),
                   probs=torch.empty(seqs * cfg.kv_heads, group, S, S, **e))
        if cfg.mlp == "swiglu":
            out["gu"] = torch.empty(tokens, 2 * cfg.ffn, **e)
        else:
            out["pre"] = torch.empty(tokens, cfg.ffn, **e)
        if cfg.sandwich:
            out["t_f"] = torch.empty(tokens, cfg.d, **e)
        if cfg.qk_norm:
            out["qk"] = torch.empty(tokens, cfg.qk_width, **e)
    return out


def workspace(cfg: DecoderConfig, tokens: int, device) -> dict:
    e = dict(dtype=torch.float32, device=device)
    group = cfg.heads // cfg.kv_heads
    seqs = tokens // cfg.seq_len
    out = {"h": torch.empty(tokens, cfg.d, **e), "qkv": torch.empty(tokens, cfg.qkv_width, **e),
           "attn": torch.empty(tokens, cfg.d, **e), "a": torch.empty(tokens, cfg.ffn, **e),
           "scores": torch.empty(seqs * cfg.kv_heads, group, cfg.seq_len, cfg.seq_len, **e),
           "tmp_d": torch.empty(tokens, cfg.d, **e), "rope": rope_tables(cfg, device),
           "streams": side_streams(cfg, tokens, device)}
    if cfg.mlp == "swiglu":
        out["gu"] = torch.empty(tokens, 2 * cfg.ffn, **e)
    return out
