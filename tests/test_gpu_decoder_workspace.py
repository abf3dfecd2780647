"""The decoder's buffers and switches: no layer's scratch holds what nothing
reads, a backward pass refuses scratch made for the other kind of checkpoint,
and the switches of forward reach sandwich and checkpointed layers."""
import pytest
import torch

from verifiable_repops_gemm_gb300 import decoder, inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
KINDS = {"llama": dict(mlp="swiglu"), "gelu": dict(mlp="gelu"),
         "sandwich": dict(mlp="swiglu", post_norm=True, gated=True, residual_scale=0.5),
         "sandwich_gelu": dict(mlp="gelu", post_norm=True, gated=True, residual_scale=0.5),
         "gated": dict(mlp="swiglu", gated=True), "scaled": dict(mlp="gelu", residual_scale=0.25)}


def config(kind):
    return decoder.DecoderConfig(d=128, heads=4, kv_heads=2, ffn=192, seq_len=24, **KINDS[kind])


def layer(kind, seqs=2):
    cfg = config(kind)
    w = decoder.init_weights(cfg, 7, DEV)
    return cfg, w, inputs.normal((seqs * cfg.seq_len, cfg.d), 1.0, 8, DEV)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int32), b.contiguous().view(torch.int32))


def tensors(d):
    return [t for t in d.values() if torch.is_tensor(t)]


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_scratch_holds_nothing_that_is_not_read(rp, kind):
    cfg, w, x = layer(kind)
    T = x.shape[0]
    ws = decoder.workspace(cfg, T, DEV)
    assert "pre" not in ws
    # the buffers that a backward pass from 8-bit checkpoints does not need share
    # those that it does
    b32, b8 = decoder.backward_workspace(cfg, T, DEV), decoder.backward_workspace(cfg, T, DEV, bits=8)
    stores = {t.untyped_storage().data_ptr(): t.untyped_storage().nbytes() for t in tensors(b8)}
    needs = {"t_ffn": cfg.ffn, "t_d": cfg.d, "dqkv": cfg.qkv_width, "h": cfg.d, "a": cfg.ffn, "qkv": cfg.qkv_width,
             "attn": cfg.d, ("gu" if cfg.mlp == "swiglu" else "pre"): cfg.ffn * (2 if cfg.mlp == "swiglu" else 1)}
    if cfg.sandwich:
        needs.update(t_e=cfg.d, t_f=cfg.d)
    scores = 2 * (T // cfg.seq_len) * cfg.heads * cfg.seq_len ** 2
    assert sum(stores.values()) == 4 * (T * sum(needs.values()) + scores)
    # every 8-bit pass runs in them, and a binary32 one in scratch made for 8 bits
    save8 = decoder.activations(cfg, T, DEV, bits=8)
    y = decoder.forward(x.clone(), w, cfg, work=ws, save=save8)
    assert same(y, decoder.forward(x.clone(), w, cfg))
    save = decoder.activations(cfg, T, DEV)
    dy = inputs.normal(x.shape, 1.0, 9, DEV)
    got = []
    for work in (b32, b8):
        decoder.forward(x.clone(), w, cfg, work=ws, save=save)
        dx, g = decoder.backward(dy.clone(), w, cfg, save, work=work)
        got.append((dx.clone(), {k: v.clone() for k, v in g.items()}))
    assert same(got[0][0], got[1][0]) and all(same(got[0][1][k], got[1][1][k]) for k in got[0][1])


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_backward_refuses_scratch_without_the_buffers_of_8_bits(rp, kind):
    cfg, w, x = layer(kind)
    save = decoder.activations(cfg, x.shape[0], DEV, bits=8)
    decoder.forward(x.clone(), w, cfg, save=save)
    dy = inputs.normal(x.shape, 1.0, 9, DEV)
    keep = dy.clone()
    with pytest.raises(ValueError, match="bits=8"):
        decoder.backward(dy, w, cfg, save, work=decoder.backward_workspace(cfg, x.shape[0], DEV))
    assert same(dy, keep)                                 # nothing was done to it


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("bits", [0, 32, 8])
def test_separate_steps_give_the_same_bits(rp, monkeypatch, kind, bits):
    """fused=False: the residual sums (and in a sandwich layer the edges' norm, gate
    and scale) as steps of their own."""
    cfg, w, x = layer(kind)

    def run(fused):
        save = decoder.activations(cfg, x.shape[0], DEV, bits=bits) if bits else None
        y = decoder.forward(x.clone(), w, cfg, save=save, fused=fused)
        kept = []
        for name, v in sorted(save.items()) if save else []:
            if name == "probs":                           # defined below the diagonal only
                continue
            kept += [t for t in (v if isinstance(v, tuple) else (v,)) if torch.is_tensor(t)]
        return y, kept

    want, kept = run(True)
    if cfg.sandwich:
        def no_edge(*a, **k):
            raise AssertionError("the fused edge ran")
        monkeypatch.setattr(decoder, "rmsnorm_residual", no_edge)
    else:
        real = decoder.gemm_batched

        def no_residual(*a, **k):
            assert cfg.mlp == "gelu" and bits or k.get("residual") is None, "a fused residual sum ran"
            return real(*a, **k)
        monkeypatch.setattr(decoder, "gemm_batched", no_residual)
    got, kept2 = run(False)
    assert same(got, want) and len(kept) == len(kept2)
    for a, b in zip(kept, kept2):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_gelu_in_the_products_epilogue_in_a_sandwich_layer(rp, monkeypatch):
    cfg, w, x = layer("sandwich_gelu")
    want = decoder.forward(x.clone(), w, cfg)

    def no_gelu(*a, **k):
        raise AssertionError("gelu ran as a kernel of its own")
    monkeypatch.setattr(decoder, "gelu", no_gelu)
    assert same(decoder.forward(x.clone(), w, cfg, gelu_epilogue=True), want)
