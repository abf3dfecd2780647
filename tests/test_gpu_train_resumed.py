"""An optimiser built again from what was kept of another one; the seed of 8-bit
moments; and the backward of normed heads from 8-bit rows, bit for bit against the
binary32 one on the same rows restored."""
import math

import pytest
import torch

from verifiable_repops_gemm_gb300 import decoder, merkle_sha256, train

from test_gpu_decoder_i8 import restored, same
from test_gpu_language_model import CFGS, DEV, T, VOCAB, batch, contributions

pytestmark = pytest.mark.gpu


def roots(model, opt):
    return {k: bytes(t.cpu().numpy()) for k, t in dict(opt.roots(), theta=merkle_sha256(model.theta)).items()}


def trained(bits, seed, data, at=None):
    """(model, optimiser) after a step on each of `data`; `at`: (theta, state, steps) to
    go on from."""
    cfg = CFGS["adjacent"]
    model = train.Model(cfg, 1, DEV, seed=5, vocab=VOCAB)
    opt = train.AdamW(model, 1e-3, bits=bits, seed=seed)
    ws = train.Workspace(model, T, DEV)
    if at is not None:
        theta, state, opt.steps = at
        model.theta.copy_(theta)
        for k, t in opt.state.items():
            t.copy_(state[k])
    for d in data:
        train.train_step(model, contributions(10 * d, cfg), 0.0, ws, optimizer=opt)
    return model, opt


@pytest.mark.parametrize("bits", [32, 8])
def test_a_run_goes_on_from_what_was_kept(rp, bits):
    """theta, the moments' buffers (whose roots are committed) and the count of steps are
    all that a run changes: with the constructor's arguments they give its next steps."""
    model, opt = trained(bits, 3, (0, 1))
    kept = model.theta.clone(), {k: t.clone() for k, t in opt.state.items()}, opt.steps
    assert kept[2] == 2
    went_on = roots(*trained(bits, 3, (0, 1, 2, 3)))
    assert roots(*trained(bits, 3, (2, 3), kept)) == went_on
    # the count is one of them: equal roots alone do not fix what comes next
    assert roots(*trained(bits, 3, (2, 3), kept[:2] + (0,)))["theta"] != went_on["theta"]


def test_another_seed_rounds_8_bit_moments_otherwise(rp):
    a, b, c = (roots(*trained(8, seed, (0,))) for seed in (3, 3, 4))
    assert a == b and all(a[k] != c[k] for k in ("m", "v")) and a["theta"] == c["theta"]
    assert roots(*trained(32, 3, (0,))) == roots(*trained(32, 4, (0,)))


@pytest.mark.parametrize("name", ["halves", "adjacent", "no_rotation", "sandwich"])
def test_normed_heads_from_8_bit_checkpoints(rp, name):
    """Every gradient and dx are the binary32 backward's on the restored rows, and the
    gains' those of head_norm_rope_backward on the restored heads."""
    cfg = CFGS[name]
    w = decoder.init_weights(cfg, 7, DEV)
    x = batch(8, cfg)[0]
    dy = torch.randn(T, cfg.d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(9)) * 1e-2
    save = decoder.activations(cfg, T, DEV, bits=8)
    decoder.forward(x.clone(), w, cfg, save=save)
    before = rp.dequantize_rows(*save["qkv"], group=decoder.CHECKPOINT_GROUP)
    seen = {}
    turn_back = decoder._rotate_backward

    def watched(dqkv, qk, *args):
        seen["qk"], seen["d"] = qk.clone(), dqkv.clone()
        turn_back(dqkv, qk, *args)
        seen["dx"] = dqkv.clone()

    decoder._rotate_backward = watched
    try:
        dx, g = decoder.backward(dy.clone(), w, cfg, save)
    finally:
        decoder._rotate_backward = turn_back
    heads, width = cfg.heads + cfg.kv_heads, cfg.qk_width
    assert same(seen["qk"], before[:, :width]) and heads * cfg.d_head == width
    tables = decoder.rope_tables(cfg, DEV) or (None, None)
    d, gq, gk = rp.head_norm_rope_backward(seen["d"][:, :width], before[:, :width], cfg.heads, cfg.kv_heads, *tables,
                                           q_gain=w["gq"], k_gain=w["gk"], eps=cfg.eps, layout=cfg.rope_layout,
                                           period=cfg.seq_len)
    assert same(g["gq"], gq) and same(g["gk"], gk) and same(seen["dx"][:, :width], d)
    assert same(seen["dx"][:, width:], seen["d"][:, width:])
    # the whole layer: qkv is kept before the heads' norms, the others as in any layer
    ws = decoder.backward_workspace(cfg, T, DEV, bits=8)
    normed = before.clone()
    decoder._rotate(normed, w, cfg, ws["rope"])
    kept = dict(save, qkv=rp.quantize_rows(normed, group=decoder.CHECKPOINT_GROUP))
    full = restored(rp, kept, w, cfg)
    out = torch.empty(T, cfg.d, device=DEV)
    decoder.attention(normed, cfg, out, None, probs=full["probs"])
    full.update(qkv=normed, qk=before[:, :width].contiguous())
    want_dx, want = decoder.backward(dy.clone(), w, cfg, full)
    assert same(dx, want_dx) and sorted(g) == sorted(w) == sorted(want)
    for k in want:
        assert same(g[k], want[k]), k
    assert math.isfinite(float(dx.abs().sum())) and bool(dx.any())
