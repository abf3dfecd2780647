"""The decoder layer with sandwich blocks, 8-bit checkpoints and 8-bit weights:
the new operators as a layer and a training step use them together.

Sandwich layers against the separate operators (bit for bit) and a binary64
autograd of the same layer; the backward from 8-bit checkpoints against the
binary32 backward on the restored activations (bit for bit); 8-bit weight
products against their own steps; the training step with 8-bit checkpoints
reproducible to its root."""
import dataclasses
import math

import pytest
import torch

from verifiable_repops_gemm_gb300 import decoder, train

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BASE = decoder.DecoderConfig(d=256, heads=4, kv_heads=2, ffn=512, seq_len=64)
SANDWICH = dataclasses.replace(BASE, post_norm=True, gated=True, residual_scale=0.5)
CONFIGS = {"llama": BASE, "gelu": dataclasses.replace(BASE, mlp="gelu"), "sandwich": SANDWICH,
           "sandwich_gelu": dataclasses.replace(SANDWICH, mlp="gelu"),
           "gated": dataclasses.replace(BASE, gated=True), "scaled": dataclasses.replace(BASE, residual_scale=0.25)}


def data(cfg, seqs, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    T = seqs * cfg.seq_len
    return (torch.randn(T, cfg.d, generator=g, device=DEV), torch.randn(T, cfg.d, generator=g, device=DEV) * 1e-2,
            decoder.init_weights(cfg, seed + 1, DEV))


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int32), b.contiguous().view(torch.int32))


@pytest.mark.parametrize("name", ["sandwich", "sandwich_gelu", "gated", "scaled"])
def test_sandwich_forward_is_the_separate_operators(rp, name):
    cfg = CONFIGS[name]
    x, _, w = data(cfg, 2, 1)
    got = decoder.forward(x.clone(), w, cfg)
    save = decoder.activations(cfg, x.shape[0], DEV)
    assert same(decoder.forward(x.clone(), w, cfg, save=save), got)
    assert same(decoder.forward(x.clone(), w, cfg, save=decoder.activations(cfg, x.shape[0], DEV, bits=8)), got)

    def edge(x, f, k):
        p = rp.rmsnorm_rows(f, w["p%d" % k], cfg.eps) if cfg.post_norm else f
        t = p * w["a%d" % k] if cfg.gated else p
        return x + t * cfg.residual_scale

    x1 = edge(x, save["f1"], 1)
    assert same(x1, save["x1"])
    h2 = rp.rmsnorm_rows(x1, w["g2"], cfg.eps)
    assert same(h2, save["h2"])
    assert same(edge(x1, save["f2"], 2), got)


def layer64(x, w, cfg):
    """The layer in binary64 from elementary torch operations."""
    T, S, dh, H, kv = x.shape[0], cfg.seq_len, cfg.d_head, cfg.heads, cfg.kv_heads

    def norm(v, g):
        return v / (v.square().mean(1, keepdim=True) + cfg.eps).sqrt() * g

    def rot(t):
        n = t.shape[1]
        freq = torch.exp(-torch.arange(dh // 2, dtype=torch.float64, device=t.device) / (dh // 2) * math.log(cfg.rope_base))
        a = (torch.arange(T, device=t.device) % S).double()[:, None] * freq
        c, s = a.cos()[:, None, :], a.sin()[:, None, :]
        p = t.reshape(T, n, dh // 2, 2)
        return torch.stack((p[..., 0] * c - p[..., 1] * s, p[..., 0] * s + p[..., 1] * c), -1).reshape(T, n, dh)

    def edge(x, f, k):
        if cfg.post_norm:
            f = norm(f, w["p%d" % k])
        if cfg.gated:
            f = f * w["a%d" % k]
        return x + cfg.residual_scale * f

    qkv = norm(x, w["g1"]) @ w["w_qkv"]
    q = rot(qkv[:, :cfg.d].reshape(T, H, dh))
    k = rot(qkv[:, cfg.d:cfg.d + kv * dh].reshape(T, kv, dh)).repeat_interleave(H // kv, 1)
    v = qkv[:, cfg.d + kv * dh:].reshape(T, kv, dh).repeat_interleave(H // kv, 1)
    q, k, v = (t.reshape(T // S, S, H, dh).transpose(1, 2) for t in (q, k, v))
    s = q @ k.transpose(2, 3) / math.sqrt(dh)
    s = s.masked_fill(torch.ones(S, S, dtype=torch.bool, device=x.device).triu(1), float("-inf"))
    attn = (s.softmax(3) @ v).transpose(1, 2).reshape(T, cfg.d)
    x = edge(x, attn @ w["w_o"], 1)
    h = norm(x, w["g2"])
    if cfg.mlp == "swiglu":
        gu = h @ w["w_gu"]
        g, u = gu[:, :cfg.ffn], gu[:, cfg.ffn:]
        f = (g * torch.sigmoid(g) * u) @ w["w_down"]
    else:
        a = h @ w["w_up"] + w["b_up"]
        f = (0.5 * a * (1 + torch.erf(a / math.sqrt(2.0)))) @ w["w_down"] + w["b_down"]
    return edge(x, f, 2)


# A product's chain of n terms is off by at most n half-steps of the sum of its
# terms' magnitudes, which for these random operands is about sqrt(n) times the
# sum: n^1.5 * 2^-24 of it.  A gradient passes at most eight products of at most
# 512 terms (128 tokens, 256, 512, 768 columns below 1.1 of that) and norms and
# softmaxes well below one of them: 8 * 1.1 * 512^1.5 * 2^-24 = 6.1e-3 of its norm.
LAYER_BOUND = 8 * 1.1 * 512 ** 1.5 * 2.0 ** -24


@pytest.mark.parametrize("name", list(CONFIGS))
def test_gradients_against_binary64(rp, name):
    cfg = CONFIGS[name]
    x, dy, w = data(cfg, 2, 10)
    save = decoder.activations(cfg, x.shape[0], DEV)
    y = decoder.forward(x.clone(), w, cfg, save=save)
    dx, g = decoder.backward(dy.clone(), w, cfg, save)
    xd = x.double().requires_grad_()
    wd = {k: v.double().requires_grad_() for k, v in w.items()}
    yd = layer64(xd, wd, cfg)
    (yd * dy.double()).sum().backward()
    assert (y.double() - yd).norm() <= LAYER_BOUND * yd.norm()
    assert (dx.double() - xd.grad).norm() <= LAYER_BOUND * xd.grad.norm()
    assert sorted(g) == sorted(w)
    for k in w:
        assert g[k].shape == w[k].shape
        assert (g[k].double() - wd[k].grad).norm() <= LAYER_BOUND * wd[k].grad.norm(), k


def restored(rp, save, w, cfg):
    """The binary32 activations the 8-bit ones stand for, with everything
    backward recomputes computed from them by the forward's operators."""
    r = {k: rp.dequantize_rows(*v, group=decoder.CHECKPOINT_GROUP) for k, v in save.items() if k != "bits"}
    r["h1"] = rp.rmsnorm_rows(r["x0"], w["g1"], cfg.eps)
    r["h2"] = rp.rmsnorm_rows(r["x1"], w["g2"], cfg.eps)
    if cfg.mlp == "swiglu":
        r["a"] = rp.swiglu(r["g"], r["u"])
        r["gu"] = torch.cat((r.pop("g"), r.pop("u")), 1)
    else:
        r["a"] = rp.gelu(r["pre"])
    T = r["x0"].shape[0]
    out = torch.empty(T, cfg.d, device=DEV)
    S, kv = cfg.seq_len, cfg.kv_heads
    r["probs"] = torch.zeros(T // S * kv, cfg.heads // kv, S, S, device=DEV)
    decoder.attention(r["qkv"], cfg, out, None, probs=r["probs"])
    return r


@pytest.mark.parametrize("name", list(CONFIGS))
def test_backward_from_8_bit_checkpoints(rp, name):
    cfg = CONFIGS[name]
    x, dy, w = data(cfg, 2, 20)
    save = decoder.activations(cfg, x.shape[0], DEV, bits=8)
    decoder.forward(x.clone(), w, cfg, save=save)
    q, s = rp.quantize_rows(x, group=decoder.CHECKPOINT_GROUP)
    assert torch.equal(save["x0"][0], q) and torch.equal(save["x0"][1], s)
    dx, g = decoder.backward(dy.clone(), w, cfg, save)
    want_dx, want = decoder.backward(dy.clone(), w, cfg, restored(rp, save, w, cfg))
    assert same(dx, want_dx)
    assert sorted(g) == sorted(w) == sorted(want)
    for k in want:
        assert same(g[k], want[k]), k
    # a second pass from the same checkpoints: they are not consumed
    grads = {k: torch.full_like(v, 7.0) for k, v in w.items()}
    dx2, g2 = decoder.backward(dy.clone(), w, cfg, save, grads=grads)
    assert same(dx2, dx) and all(g2[k] is grads[k] and same(grads[k], g[k]) for k in g)


def test_8_bit_checkpoints_are_smaller():
    def size(save):
        return sum(t.numel() * t.element_size() for v in save.values() if not isinstance(v, int) for t in (v if isinstance(v, tuple) else (v,)))

    full, kept = (size(decoder.activations(BASE, 128, DEV, bits=b)) for b in (32, 8))
    # x0, qkv, attn, x1, g and u of 3 * 256 + 512 + 2 * 512 columns at 1 + 4/128
    # bytes, against those, h1, h2 and a at 4 and 2 * 4 heads' 64 x 64 probabilities
    assert kept == 128 * (3 * 256 + 512 + 2 * 512) * 33 // 32
    assert full == 128 * (5 * 256 + 512 + 3 * 512) * 4 + 2 * 4 * 64 * 64 * 4


@pytest.mark.parametrize("name", list(CONFIGS))
def test_forward_with_8_bit_weights(rp, name):
    cfg = CONFIGS[name]
    x, _, w = data(cfg, 2, 30)
    w8 = decoder.quantize_weights(w, cfg)
    assert sorted(w8) == sorted(k for k in w if k in decoder.WEIGHT_MATRICES)
    got = decoder.forward_i8(x.clone(), w, w8, cfg)

    def product(rows, name):
        q, s = rp.quantize_rows(rows)
        return rp.gemm_i8(q, w8[name][0].t(), s.view(-1), w8[name][1])

    def edge(x, f, k):
        p = rp.rmsnorm_rows(f, w["p%d" % k], cfg.eps) if cfg.post_norm else f
        t = p * w["a%d" % k] if cfg.gated else p
        return x + t * cfg.residual_scale

    qkv = product(rp.rmsnorm_rows(x, w["g1"], cfg.eps), "w_qkv")
    cos, sin = decoder.rope_tables(cfg, DEV)
    rp.rope(qkv, cfg.heads + cfg.kv_heads, cos, sin, period=cfg.seq_len)
    attn = torch.empty_like(x)
    decoder.attention(qkv, cfg, attn, torch.empty(2 * cfg.kv_heads, 2, 64, 64, device=DEV))
    x1 = edge(x, product(attn, "w_o"), 1)
    h = rp.rmsnorm_rows(x1, w["g2"], cfg.eps)
    if cfg.mlp == "swiglu":
        gu = product(h, "w_gu")
        f = product(rp.swiglu(gu[:, :cfg.ffn], gu[:, cfg.ffn:]), "w_down")
    else:
        f = product(rp.gelu(product(h, "w_up") + w["b_up"]), "w_down") + w["b_down"]
    assert same(got, edge(x1, f, 2))
    # each 8-bit product is within its operands' steps, 1/254 of their largest
    # values each: a few per cent of the layer's change, never a different result
    y = decoder.forward(x.clone(), w, cfg)
    assert (got - y).norm() <= 0.1 * (y - x).norm()


@pytest.mark.parametrize("name", ["llama", "sandwich"])
def test_training_step_with_8_bit_checkpoints_is_reproducible(rp, name):
    cfg = CONFIGS[name]
    T = 2 * cfg.seq_len
    g = torch.Generator(device=DEV).manual_seed(40)
    contribs = [(did, torch.randn(T, cfg.d, generator=g, device=DEV), torch.randn(T, cfg.d, generator=g, device=DEV) * 1e-2)
                for did in (b"did:zoo:b", b"did:zoo:a", b"did:zoo:c")]
    roots = set()
    for order in (contribs, contribs[::-1]):
        model = train.Model(cfg, 2, DEV, seed=41)
        ws = train.Workspace(model, T, DEV, checkpoint_bits=8)
        before = model.theta.clone()
        for _ in range(2):
            root, _ = train.train_step(model, order, 1e-2, ws)
        assert torch.isfinite(model.theta).all() and not torch.equal(model.theta, before)
        roots.add(bytes(root.cpu().numpy()))
    assert len(roots) == 1
