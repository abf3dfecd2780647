"""The new ends of a training step together: a model with normed and rotated query
and key heads (halves, part of a head, scaled frequencies), the loss of given
tokens and AdamW, through decoder.py and train.py -- against a statement in
binary64 with automatic gradients, bit for bit across contributors' orders,
replays and ways of keeping activations, and the update against its formula."""
import itertools
import math

import numpy as np
import pytest
import torch

from verifiable_repops_gemm_gb300 import decoder, train

import adamw_ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
VOCAB = 333
BASE = dict(d=128, heads=4, kv_heads=2, ffn=256, seq_len=48, rope_base=10000.0)
CFGS = {"halves": decoder.DecoderConfig(**BASE, qk_norm=True, rope_layout="halves", rope_dim=16, rope_factor=4.0,
                                        rope_original=64.0),
        "adjacent": decoder.DecoderConfig(**BASE, qk_norm=True),
        "no_norm": decoder.DecoderConfig(**BASE, rope_layout="halves"),
        "no_rotation": decoder.DecoderConfig(**{**BASE, "rope_base": 0.0}, qk_norm=True),
        "sandwich": decoder.DecoderConfig(**BASE, qk_norm=True, rope_dim=8, post_norm=True, gated=True, mlp="gelu")}
T = 96


def batch(seed, cfg):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, cfg.d, generator=g, device=DEV)
    t = torch.randint(0, VOCAB, (T,), generator=g, device=DEV)
    t[5] = t[60] = -100
    return x, t


def norm(v, gain, eps):
    return v / (v.square().mean(-1, keepdim=True) + eps).sqrt() * gain


def layer64(x, w, cfg):
    """One layer in binary64."""
    S, dh, H, kv = cfg.seq_len, cfg.d_head, cfg.heads, cfg.kv_heads
    qkv = norm(x, w["g1"], cfg.eps) @ w["w_qkv"]
    q, k, v = qkv.split([H * dh, kv * dh, kv * dh], 1)
    q, k, v = q.view(-1, S, H, dh), k.view(-1, S, kv, dh), v.view(-1, S, kv, dh)
    if cfg.qk_norm:
        q, k = norm(q, w["gq"], cfg.eps), norm(k, w["gk"], cfg.eps)
    if cfg.rope_base:
        n = (cfg.rope_dim or dh) // 2
        f = torch.exp(-torch.arange(n, dtype=torch.float64, device=DEV) / n * math.log(cfg.rope_base))
        if cfg.rope_factor != 1.0:
            r = ((cfg.rope_original * f / (2 * math.pi) - 1.0) / 3.0).clamp(0, 1)
            f = f / cfg.rope_factor * (1 - r) + f * r
        ang = torch.arange(S, dtype=torch.float64, device=DEV)[:, None] * f
        c, s = ang.cos()[:, None], ang.sin()[:, None]

        def turn(h):
            if cfg.rope_layout == "halves":
                a, b, rest = h[..., :n], h[..., n:2 * n], h[..., 2 * n:]
                return torch.cat([a * c - b * s, a * s + b * c, rest], -1)
            a, b, rest = h[..., 0:2 * n:2], h[..., 1:2 * n:2], h[..., 2 * n:]
            return torch.cat([torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2), rest], -1)

        q, k = turn(q), turn(k)
    k, v = (t.repeat_interleave(H // kv, 2) for t in (k, v))
    sc = torch.einsum("bihd,bjhd->bhij", q, k) / dh ** 0.5
    sc = sc.masked_fill(torch.ones(S, S, dtype=torch.bool, device=DEV).triu(1), -math.inf)
    f1 = torch.einsum("bhij,bjhd->bihd", sc.softmax(-1), v).reshape(x.shape) @ w["w_o"]

    def edge(x, f, i):
        p = norm(f, w["p%d" % i], cfg.eps) if cfg.post_norm else f
        return x + cfg.residual_scale * (p * w["a%d" % i] if cfg.gated else p)

    x = edge(x, f1, 1)
    h = norm(x, w["g2"], cfg.eps)
    if cfg.mlp == "swiglu":
        g, u = (h @ w["w_gu"]).chunk(2, 1)
        f2 = (torch.nn.functional.silu(g) * u) @ w["w_down"]
    else:
        f2 = torch.nn.functional.gelu(h @ w["w_up"] + w["b_up"]) @ w["w_down"] + w["b_down"]
    return edge(x, f2, 2)


def gradient64(model, x, t):
    """(logp, flat gradient) of the mean negative log probability in binary64."""
    theta = model.theta.double().requires_grad_()
    views = model.views(theta)
    h = x.double()
    for layer in range(model.layers):
        h = layer64(h, views[layer], model.cfg)
    out = views[model.layers]
    lp = torch.log_softmax(norm(h, out["g_out"], model.cfg.eps) @ out["w_out"], 1)
    logp = torch.where(t >= 0, lp.gather(1, t.clamp_min(0)[:, None])[:, 0], 0.0)
    (-logp.sum() / (t >= 0).sum()).backward()
    return logp.detach(), theta.grad


@pytest.mark.parametrize("name", sorted(CFGS))
def test_gradient_against_binary64(rp, name):
    """Every weight's gradient within 2e-5 of its norm: chains of at most 333 products
    each rounded twice (2 * sqrt(333) * 2^-24 = 2.2e-6 where roundings are independent),
    about ten of them one after another."""
    cfg = CFGS[name]
    model = train.Model(cfg, 2, DEV, seed=3, vocab=VOCAB)
    x, t = batch(4, cfg)
    ws = train.Workspace(model, T, DEV)
    g, logp = train.token_gradient(model, x, t, model.gradient_buffer(), ws)
    want_lp, want = gradient64(model, x, t)
    assert (logp.double() - want_lp).abs().max() <= 2e-5
    assert logp[5] == 0 and logp[60] == 0
    for layer, key, off, shape in model.slots:
        a, b = g[off:off + math.prod(shape)].double(), want[off:off + math.prod(shape)]
        assert (a - b).norm() <= 2e-5 * b.norm(), (layer, key)


def test_upstream_gradients_leave_the_vocabulary_at_zero(rp):
    """A buffer that held another gradient before: every weight's part is written."""
    cfg = CFGS["adjacent"]
    model = train.Model(cfg, 1, DEV, seed=3, vocab=VOCAB)
    ws = train.Workspace(model, T, DEV)
    dy = torch.randn(T, cfg.d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(12))
    clean = train.contributor_gradient(model, batch(4, cfg)[0], dy, model.gradient_buffer(), ws)
    used = train.contributor_gradient(model, batch(4, cfg)[0], dy, model.gradient_buffer().fill_(float("nan")), ws)
    for layer, key, off, shape in model.slots:
        part = slice(off, off + math.prod(shape))
        assert torch.equal(clean[part], used[part]), (layer, key)
        assert layer < model.layers or not used[part].any()


def test_a_refused_step_counts_for_nothing(rp):
    cfg = CFGS["adjacent"]
    model = train.Model(cfg, 1, DEV, seed=3)
    opt = train.AdamW(model, 1e-3)
    g = model.gradient_buffer()
    with pytest.raises(Exception):
        opt.step([g, g], [0, 0])
    assert opt.steps == 0
    opt.step([g, g], [1, 0])
    assert opt.steps == 1


def contributions(seed, cfg):
    return [(did, *batch(seed + i, cfg)) for i, did in enumerate((b"did:zoo:charlie", b"did:zoo:alice", b"did:zoo:bob"))]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("checkpoint", [32, 8])
def test_steps_do_not_depend_on_arrival(rp, bits, checkpoint):
    """Two steps of three contributors in every order of arrival: one root of theta,
    one of each moment; another seed rounds 8-bit moments otherwise."""
    cfg = CFGS["halves"]
    got = set()
    for perm in itertools.permutations(range(3)):
        model = train.Model(cfg, 2, DEV, seed=5, vocab=VOCAB)
        opt = train.AdamW(model, 1e-3, bits=bits)
        ws = train.Workspace(model, T, DEV, checkpoint_bits=checkpoint)
        for step in range(2):
            c = contributions(10 * step, cfg)
            root, order = train.train_step(model, [c[i] for i in perm], 0.0, ws, optimizer=opt)
        roots = opt.roots()
        assert set(roots) == ({"m", "v"} if bits == 32 else {"m", "v", "m_scales", "v_scales"})
        got.add((root.cpu().numpy().tobytes(),) + tuple(roots[k].cpu().numpy().tobytes() for k in sorted(roots)))
    assert len(got) == 1
    assert torch.isfinite(model.theta).all()


def test_update_is_adamw_of_the_mean_gradient(rp):
    cfg = CFGS["adjacent"]
    model = train.Model(cfg, 1, DEV, seed=6, vocab=VOCAB)
    opt = train.AdamW(model, 2e-3)
    ws = train.Workspace(model, T, DEV)
    c = contributions(30, cfg)
    grads = [model.gradient_buffer() for _ in c]
    was = model.theta.cpu().numpy()
    _, order = train.train_step(model, c, 0.0, ws, grads=grads, optimizer=opt)
    n = model.theta.numel()
    decay = np.zeros(n, np.float32)
    for (_, _, off, shape), d in zip(model.slots, opt.decay):
        decay[off:off + math.prod(shape)] = d
    z = np.zeros(n, np.float32)
    want = adamw_ref.step(was, [grads[i].cpu().numpy() for i in order], z, z, adamw_ref.scalars(1, 2e-3, opt.betas), decay,
                          opt.betas, opt.eps)
    assert np.array_equal(model.theta.cpu().numpy().view(np.uint32), want[0].view(np.uint32))
    assert np.array_equal(opt.state["m"].cpu().numpy(), want[1])


def test_8_bit_checkpoints_give_the_gradient_of_the_restored_activations(rp):
    """qk_norm's backward from 8-bit rows: the binary32 backward's bits on the same
    rows restored."""
    cfg = CFGS["halves"]
    w = decoder.init_weights(cfg, 7, DEV)
    x = batch(8, cfg)[0]
    dy = torch.randn(T, cfg.d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(9)) * 1e-2
    save = decoder.activations(cfg, T, DEV, bits=8)
    y8 = decoder.forward(x.clone(), w, cfg, save=save)
    full = decoder.activations(cfg, T, DEV)
    y = decoder.forward(x.clone(), w, cfg, save=full)
    assert torch.equal(y, y8)                      # what is kept does not change what is computed
    restored = rp.dequantize_rows(*save["qkv"], group=decoder.CHECKPOINT_GROUP)
    dx8, g8 = decoder.backward(dy.clone(), w, cfg, save)
    # the same attention backward from the restored rows, by the separate calls
    ws = decoder.backward_workspace(cfg, T, DEV, bits=8)
    again = decoder._recomputed_attention(save, w, cfg, ws)
    assert torch.equal(again["qk"], restored[:, :cfg.qk_width])
    normed = restored.clone()
    decoder._rotate(normed, w, cfg, ws["rope"])
    assert torch.equal(again["qkv"], normed)
    dx, g = decoder.backward(dy.clone(), w, cfg, full)
    for k in g:
        assert (g8[k] - g[k]).norm() <= 0.05 * g[k].norm(), k     # 8-bit activations: under 1 percent each


def test_inference_in_8_bits_runs_with_normed_heads(rp):
    cfg = CFGS["halves"]
    w = decoder.init_weights(cfg, 7, DEV)
    x = batch(8, cfg)[0]
    y = decoder.forward(x.clone(), w, cfg)
    y8 = decoder.forward_i8(x.clone(), w, decoder.quantize_weights(w, cfg), cfg)
    assert (y8 - y).norm() <= 0.05 * y.norm()
